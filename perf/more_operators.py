"""Cases, plain forms and calls of the operators that a prompt's attention over the paged latent cache is made of.

* gather:  cached tokens of several requests read back from the paged cache (three formats) into packed bf16 rows;
* prefill: attention of packed sequences of different lengths, per-head keys and values (128 columns, 64 more of the key
           shared by the heads or absent), causal to the sequences' ends or over all keys, with log-sum-exp;
* merge:   attention outputs over several sets of keys joined by their log-sum-exps.

Packed sequences: sequence i owns rows cu[i] .. cu[i + 1] - 1.  With causal attention the last query of a sequence sees
all its keys, the one before all but the last, and so on.
"""
import math

import torch

own = False

D_LATENT, D_KEY, PAGE = 512, 576, 64
D_NOPE, D_ROPE, D_V = 128, 64, 128


def listed():
    return [
        # the cached prefixes of two short requests: the smallest calls, latency alone
        dict(name="gather_tiny", op="gather", fmt="bf16", b=2, lo=100, hi=333, first=0),
        # prefixes of 24 requests of a 656-byte cache
        dict(name="gather_prefix_656", op="gather", fmt="fp8_656", b=24, lo=1024, hi=8192, first=0),
        # one piece of long contexts (from the middle of a page on), 528-byte cache
        dict(name="gather_piece_528", op="gather", fmt="fp8_528", b=9, lo=1021, hi=1021, first=5000),
        # two short prompts, 16 heads
        dict(name="prefill_tiny", op="prefill", b=2, q_lo=100, q_hi=333, ctx_lo=0, ctx_hi=0, h=16, h_k=16, rope="shared", causal=True),
        # whole prompts, 128 heads: the ordinary case
        dict(name="prefill_prompts", op="prefill", b=2, q_lo=2048, q_hi=4096, ctx_lo=0, ctx_hi=0, h=128, h_k=128, rope="shared", causal=True),
        # one long prompt, 16 heads: the largest
        dict(name="prefill_long", op="prefill", b=1, q_lo=16384, q_hi=16384, ctx_lo=0, ctx_hi=0, h=16, h_k=16, rope="shared", causal=True),
        # many short prompts of odd lengths packed together
        dict(name="prefill_ragged", op="prefill", b=61, q_lo=1, q_hi=601, ctx_lo=0, ctx_hi=0, h=64, h_k=64, rope="shared", causal=True),
        # grouped heads without position columns
        dict(name="prefill_grouped", op="prefill", b=3, q_lo=700, q_hi=2500, ctx_lo=0, ctx_hi=0, h=64, h_k=8, rope="none", causal=True),
        # chunks of 512 new tokens over what their requests hold already
        dict(name="prefill_chunk", op="prefill", b=4, q_lo=512, q_hi=512, ctx_lo=1000, ctx_hi=7500, h=64, h_k=64, rope="shared", causal=True),
        # a few new tokens (one at least) over a piece of a long context, all of it visible
        dict(name="prefill_few", op="prefill", b=3, q_lo=1, q_hi=16, ctx_lo=8000, ctx_hi=16384, h=16, h_k=16, rope="shared", causal=False),
        # the outputs of a step's requests over two sets of keys
        dict(name="merge_step", op="merge", n=2, rows=64, h=128, d=512, f32=False),
        # the outputs of a prompt's chunk over four pieces of its context and itself
        dict(name="merge_chunk", op="merge", n=5, rows=2048, h=128, d=128, f32=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gather", "prefill", "prefill", "merge"])
    if op == "gather":
        b = _log(rng, 1, 256)
        hi = _log(rng, 1, min(16384, 196_608 // b))
        return dict(op=op, fmt=rng.choice(["bf16", "fp8_656", "fp8_528"]), b=b, lo=rng.randint(0, hi), hi=hi,
                    first=rng.choice([0, 0, _log(rng, 1, 8192)]))
    if op == "merge":
        d, h = rng.choice([64, 128, 512]), rng.choice([1, 5, 16, 64, 128])
        n = rng.choice([2, 2, _log(rng, 3, 16)])
        return dict(op=op, n=n, rows=_log(rng, 1, max(1, min(16384, 150_000_000 // (d * h * n)))), h=h, d=d, f32=rng.random() < 0.4)
    h_k, group = rng.choice([(1, 1), (16, 1), (64, 1), (128, 1), (5, 1), (8, 8), (4, 6), (2, 5), (1, 16)])
    b = rng.choice([1, 2, _log(rng, 3, 64)])
    q_hi = _log(rng, 1, 8192)
    ctx_hi = rng.choice([0, 0, _log(rng, 1, 16384)])
    causal = rng.random() < 0.7
    # pairs of query and key: those of the plain form's padded square, and those that count
    while b * h_k * group * q_hi * max(q_hi + ctx_hi, 2 * ctx_hi + q_hi * (1 if causal else 2)) > 4_200_000_000:
        b, q_hi, ctx_hi = max(1, b // 2), max(1, q_hi * 2 // 3), ctx_hi * 2 // 3
    return dict(op=op, b=b, q_lo=rng.randint(1, q_hi), q_hi=q_hi, ctx_lo=rng.randint(0, ctx_hi), ctx_hi=ctx_hi, h=h_k * group, h_k=h_k,
                rope=rng.choice(["shared", "shared", "own", "none"]), causal=causal)


# ------------------------------------------------------------------ inputs


def _starts(lens, dev):
    """[0, lens[0], lens[0] + lens[1], ...] as int32."""
    return torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(lens, 0)]).int().to(dev)


def _lens(lo, hi, b, host):
    """b lengths spread evenly over lo .. hi (hi where b is 1), in an order of the seed's: the packed rows are as many for every seed."""
    lens = torch.tensor(_spread(lo, hi, b))
    return lens[torch.randperm(b, generator=host)]


def _spread(lo, hi, b):
    return [hi - (hi - lo) * i // max(1, b - 1) for i in range(b)]


def _encode(x, fmt):
    """float32 rows -> cache rows (bf16, or bytes)."""
    if fmt == "bf16":
        return x.to(torch.bfloat16)
    if fmt == "fp8_656":
        tiles = x[..., :D_LATENT].unflatten(-1, (4, 128))
        scale = tiles.abs().amax(-1) / 448.0
        codes = (tiles / scale[..., None]).to(torch.float8_e4m3fn).flatten(-2)
        return torch.cat([codes.view(torch.uint8), scale.view(torch.uint8), x[..., D_LATENT:].to(torch.bfloat16).contiguous().view(torch.uint8)], -1)
    blocks = x.unflatten(-1, (16, 32))
    mant, expo = torch.frexp(blocks.abs().amax(-1) / 448.0)  # the smallest power of two at or above the ratio
    expo = torch.where(mant == 0.5, expo - 1, expo)
    codes = torch.ldexp(blocks, -expo[..., None]).to(torch.float8_e4m3fn).flatten(-2)
    return torch.cat([codes.view(torch.uint8), (expo + 127).to(torch.uint8)], -1)


def _width(fmt):
    return D_LATENT if fmt == "fp8_528" else D_KEY


def _gather_inputs(case, dev, host, g):
    b = case["b"]
    lens = _lens(case["lo"], case["hi"], b, host)
    first = torch.randint(case["first"] // 2, case["first"] + 1, (b,), generator=host)
    slots = torch.arange((case["first"] + case["hi"] + PAGE - 1) // PAGE)[None]
    live = (slots * PAGE < (first + lens)[:, None]) & (slots >= (first // PAGE)[:, None])  # pages that hold a token of the call
    pages = int(live.sum()) + 1
    number = torch.cumsum(live.reshape(-1).int(), 0).reshape(live.shape) - 1
    table = torch.where(live, torch.randperm(pages, generator=host)[number.clamp(min=0)], -1).int()
    rows = torch.randn(pages, PAGE, _width(case["fmt"]), generator=g, device=dev)
    total = int(lens.sum())
    return dict(cu=_starts(lens, dev), first=first.int().to(dev) if case["first"] else None, table=table.to(dev), cache=_encode(rows, case["fmt"]),
                total=total, out=torch.zeros(total, _width(case["fmt"]), dtype=torch.bfloat16, device=dev))


def _prefill_inputs(case, dev, host, g):
    q_lens = _lens(case["q_lo"], case["q_hi"], case["b"], host)
    k_lens = _lens(case["ctx_lo"], case["ctx_hi"], case["b"], host)
    if case["causal"] or case["ctx_hi"] == 0:
        k_lens = k_lens + q_lens
    nq, nk, h, h_k = int(q_lens.sum()), int(k_lens.sum()), case["h"], case["h_k"]
    make = lambda *shape: torch.randn(*shape, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
    st = dict(cu_q=_starts(q_lens, dev), cu_k=_starts(k_lens, dev), nq=nq, nk=nk, k_rope=None)
    if case["rope"] == "none":
        st["q"], st["k"], st["v"] = 1.5 * make(nq, h, D_NOPE), make(nk, h_k, D_NOPE), make(nk, h_k, D_V)
    else:
        st["q"] = 1.5 * make(nq, h, D_NOPE + D_ROPE)
        if case["rope"] == "shared":  # keys and values beside each other as a projection leaves them, position columns of gathered rows
            both = make(nk, h_k, D_NOPE + D_V)
            st["k"], st["v"], st["k_rope"] = both[..., :D_NOPE], both[..., D_NOPE:], make(nk, D_KEY)[:, D_LATENT:]
        else:  # whole keys, head by head
            keys = make(nk, h_k, D_NOPE + D_ROPE)
            st["k"], st["k_rope"], st["v"] = keys[..., :D_NOPE], keys[..., D_NOPE:], make(nk, h_k, D_V)
    st["scale"] = 1.0 / math.sqrt(st["q"].shape[-1])
    return st


def _merge_inputs(case, dev, g):
    n, rows, h, d = case["n"], case["rows"], case["h"], case["d"]
    lses = 6.0 + 1.5 * torch.randn(n, h, rows, generator=g, device=dev)
    none = torch.rand(n, 1, rows, generator=g, device=dev) < 0.1  # a token that sees no key of a set
    lses = torch.where(none, -math.inf, lses)
    parts = torch.randn(n, rows, h, d, generator=g, device=dev)
    parts = torch.where(none.permute(0, 2, 1)[..., None], 0.0, parts)
    return dict(parts=parts if case["f32"] else parts.to(torch.bfloat16), lses=lses,
                out=torch.zeros(rows, h, d, dtype=torch.bfloat16, device=dev), lse=torch.zeros(h, rows, device=dev))


def _inputs(case, seed):
    dev = torch.device("cuda")
    host, g = torch.Generator().manual_seed(seed), torch.Generator(device=dev).manual_seed(seed)
    if case["op"] == "gather":
        st = _gather_inputs(case, dev, host, g)
    elif case["op"] == "prefill":
        st = _prefill_inputs(case, dev, host, g)
    else:
        st = _merge_inputs(case, dev, g)
    st["case"] = case
    st["err"] = torch.zeros(1, dtype=torch.int32, device=dev)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own and case["op"] == "prefill":  # the buffers that a serving loop holds for this shape
        from mla_decode_attention_gb300 import binding
        st["buf"] = binding.PrefillBuffers(st["nq"], st["nk"], case["b"], case["h"], case["h_k"], "cuda")
    return st


# ------------------------------------------------------------------ plain forms


def _rows_of(cu, total):
    """Sequence of every packed row, and the row's place in it."""
    row = torch.arange(total, device=cu.device)
    seq = torch.searchsorted(cu[1:].contiguous(), row.int(), right=True)
    return seq, row - cu.long()[seq]


def _gather_plain(st):
    case = st["case"]
    seq, at = _rows_of(st["cu"], st["total"])
    if st["first"] is not None:
        at = at + st["first"].long()[seq]
    rows = st["cache"].view(-1, st["cache"].shape[-1])[st["table"].long()[seq, at // PAGE] * PAGE + at % PAGE]
    if case["fmt"] == "bf16":
        return rows
    codes = rows[:, :D_LATENT].contiguous().view(torch.float8_e4m3fn).float()
    if case["fmt"] == "fp8_656":
        scale = rows[:, 512:528].contiguous().view(torch.float32)
        latent = (codes.unflatten(-1, (4, 128)) * scale[..., None]).flatten(-2).to(torch.bfloat16)
        return torch.cat([latent, rows[:, 528:].contiguous().view(torch.bfloat16)], -1)
    return (codes.unflatten(-1, (16, 32)) * torch.exp2(rows[:, 512:].float() - 127.0)[..., None]).flatten(-2).to(torch.bfloat16)


def _padded(x, cu, most):
    """Packed rows [n, h, d] -> float32 [b, h, most, d]; what is past a sequence's end is some other row."""
    at = (cu[:-1, None].long() + torch.arange(most, device=cu.device)).clamp(max=x.shape[0] - 1)
    return x[at].transpose(1, 2).float()


def _prefill_plain(st):
    case = st["case"]
    b, h, h_k = case["b"], case["h"], case["h_k"]
    cu_q, cu_k = st["cu_q"], st["cu_k"]
    n = case["q_hi"]
    m = case["ctx_hi"] + (case["q_hi"] if case["causal"] or case["ctx_hi"] == 0 else 0)
    keys = st["k"]
    if st["k_rope"] is not None:
        rope = st["k_rope"] if case["rope"] == "own" else st["k_rope"][:, None].expand(-1, h_k, -1)
        keys = torch.cat([keys, rope], -1)
    q = _padded(st["q"], cu_q, n).mul_(st["scale"]).reshape(b, h_k, (h // h_k) * n, -1)
    scores = (q @ _padded(keys, cu_k, m).transpose(-1, -2)).view(b, h_k, h // h_k, n, m)
    q_len, k_len = (cu_q[1:] - cu_q[:-1]).long()[:, None, None], (cu_k[1:] - cu_k[:-1]).long()[:, None, None]
    last = k_len - 1
    if case["causal"]:
        last = last - q_len + 1 + torch.arange(n, device=q.device)[None, :, None]
    unseen = torch.arange(m, device=q.device)[None, None] > last
    scores.masked_fill_(unseen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total))[..., 0].reshape(b, h, n)
    out = (p.view(b, h_k, -1, m) @ _padded(st["v"], cu_k, m)).view(b, h, n, D_V) / torch.where(total > 0, total, 1.0).reshape(b, h, n, 1)
    seq, at = _rows_of(cu_q, st["nq"])
    return out[seq, :, at].to(torch.bfloat16), lse[seq, :, at].T.contiguous()


def _merge_plain(st):
    lses = st["lses"]
    top = lses.amax(0)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    w = torch.exp(lses - top)
    total = w.sum(0)
    lse = top + torch.log(total)
    w = (w / torch.where(total > 0, total, 1.0)).permute(0, 2, 1)[..., None]
    return (w * st["parts"].float()).sum(0).to(torch.bfloat16), lse


# ------------------------------------------------------------------ one pass


def run(state):
    case = state["case"]
    if not own:
        return {"gather": _gather_plain, "prefill": _prefill_plain, "merge": _merge_plain}[case["op"]](state)
    from mla_decode_attention_gb300 import binding
    if case["op"] == "gather":
        formats = {"bf16": binding.MLA_KV_BF16, "fp8_656": binding.MLA_KV_FP8_656, "fp8_528": binding.MLA_KV_FP8_528}
        binding.mla_gather_kv(state["cache"], formats[case["fmt"]], state["table"], state["cu"], state["out"], starts=state["first"], err=state["err"])
        return state["out"]
    if case["op"] == "merge":
        binding.mla_merge_states(state["parts"], state["lses"], state["out"], state["lse"])
        return state["out"], state["lse"]
    buf = state["buf"]
    binding.mla_prefill(state["q"], state["k"], state["v"], state["cu_q"], state["cu_k"], state["scale"], case["causal"], buf.num_sm_parts,
                        buf.workspace, buf.out, buf.lse, k_rope=state["k_rope"], err=buf.err)
    return buf.out, buf.lse


# ------------------------------------------------------------------ work and exact values


def work(case):
    if case["op"] == "gather":
        rows = sum(_spread(case["lo"], case["hi"], case["b"]))
        token = {"bf16": 1152, "fp8_656": 656, "fp8_528": 528}[case["fmt"]]
        return {"bytes": rows * (token + 2 * _width(case["fmt"]) + 4 / PAGE) + 8 * case["b"], "flops": 0 if case["fmt"] == "bf16" else rows * D_LATENT}
    if case["op"] == "merge":
        rows, n = case["rows"] * case["h"], case["n"]
        return {"bytes": rows * (n * ((4 if case["f32"] else 2) * case["d"] + 4) + 2 * case["d"] + 4), "flops": rows * n * (2 * case["d"] + 4)}
    d = D_NOPE + (0 if case["rope"] == "none" else D_ROPE)
    h, h_k = case["h"], case["h_k"]
    q_lens, ctx = _spread(case["q_lo"], case["q_hi"], case["b"]), _spread(case["ctx_lo"], case["ctx_hi"], case["b"])
    nq, nk, both = sum(q_lens), sum(ctx), sum(q_lens) * sum(ctx) / case["b"]  # (the orders are independent)
    if case["causal"]:
        nk, pairs = nk + nq, both + sum(n * (n + 1) / 2 for n in q_lens)
    elif case["ctx_hi"] == 0:
        nk, pairs = nq, sum(n * n for n in q_lens)
    else:
        pairs = both
    rope = {"none": 0, "shared": D_ROPE, "own": h_k * D_ROPE}[case["rope"]]
    return {"bytes": nq * h * (2 * d + 2 * D_V + 4) + nk * 2 * (h_k * (D_NOPE + D_V) + rope), "flops": 2 * h * pairs * (d + D_V)}


def _exact_gather(case, st):
    """Token by token's place in the pool; e4m3 is sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    cu, table = st["cu"].tolist(), st["table"].long()
    first = st["first"].tolist() if st["first"] is not None else [0] * case["b"]
    places = [torch.zeros(0, dtype=torch.long, device=table.device)]
    for i in range(case["b"]):
        at = torch.arange(first[i], first[i] + cu[i + 1] - cu[i], device=table.device)
        places.append(table[i][torch.div(at, 64, rounding_mode="floor")] * 64 + at.remainder(64))
    rows = st["cache"].flatten(0, 1)[torch.cat(places)]
    if case["fmt"] == "bf16":
        return rows.double()
    code = torch.arange(256, device=rows.device)
    sign, e, f = 1.0 - 2.0 * (code // 128).double(), (code // 8 % 16).double(), (code % 8).double()
    value = (sign * torch.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * torch.pow(2.0, e - 7)))[rows[:, :512].long()]
    if case["fmt"] == "fp8_656":
        scale = rows[:, 512:528].contiguous().view(torch.float32).double().repeat_interleave(128, 1)
        return torch.cat([value * scale, rows[:, 528:].contiguous().view(torch.bfloat16).double()], 1)
    return value * torch.pow(2.0, rows[:, 512:].double() - 127).repeat_interleave(32, 1)


def _exact_prefill(case, st):
    """One sequence and head after another."""
    out = torch.zeros(st["nq"], case["h"], D_V, dtype=torch.float64, device="cuda")
    lse = torch.full((case["h"], st["nq"]), -math.inf, dtype=torch.float64, device="cuda")
    cu_q, cu_k, group = st["cu_q"].tolist(), st["cu_k"].tolist(), case["h"] // case["h_k"]
    for i in range(case["b"]):
        a, z, c, e = cu_q[i], cu_q[i + 1], cu_k[i], cu_k[i + 1]
        if a == z or c == e:
            continue
        see = None
        if case["causal"]:
            see = torch.ones(z - a, e - c, dtype=torch.bool, device="cuda").tril((e - c) - (z - a))
        for j in range(case["h"]):
            k = st["k"][c:e, j // group].double()
            s = st["q"][a:z, j, :D_NOPE].double() @ k.T
            if st["k_rope"] is not None:
                turned = st["k_rope"][c:e, j // group] if case["rope"] == "own" else st["k_rope"][c:e]
                s += st["q"][a:z, j, D_NOPE:].double() @ turned.double().T
            s *= st["scale"]
            if see is not None:
                s = torch.where(see, s, -math.inf)
            total = torch.logsumexp(s, 1)
            out[a:z, j] = torch.where(torch.isinf(total)[:, None], 0.0, torch.exp(s - total[:, None])) @ st["v"][c:e, j // group].double()
            lse[j, a:z] = total
    return out, lse


def exact(case, seed):
    """The definitions in 64 bits, written apart from the plain forms."""
    st = _inputs(case, seed)
    if case["op"] == "gather":
        return _exact_gather(case, st)
    if case["op"] == "prefill":
        return _exact_prefill(case, st)
    total = torch.logsumexp(st["lses"].double(), 0)
    share = torch.where(torch.isinf(total), 0.0, torch.exp(st["lses"].double() - total))
    out = torch.zeros(case["rows"], case["h"], case["d"], dtype=torch.float64, device="cuda")
    for i in range(case["n"]):
        out += share[i].T[..., None] * st["parts"][i].double()
    return out, total
