"""Cases, plain forms and calls of the operators around a windowed decode step over the paged latent cache.

* append: new tokens' latent rows, normalised and rotated, written into the paged cache (three cache formats);
* query:  RMS norm of every query head and rotation of its last 64 columns, in one pass;
* window: attention of the new tokens over the last ``window`` cached tokens and the first ``sinks`` ones.

Conventions shared by the three: ``lens[b]`` counts a request's cached tokens, the new ones included; ``new[b]`` of its
``s`` token slots hold new tokens (all of them where ``new`` is None); token j of request b sits at position
``lens[b] - new[b] + j``.  Slots with j >= new[b], or a negative position, are padding.
"""
import math

import torch

own = False

D_LATENT, D_ROPE, D_KEY, PAGE = 512, 64, 576, 64
SCALE = 1.0 / math.sqrt(192.0)
EPS = 1e-6
TOKEN_BYTES = {"bf16": 1152, "fp8_656": 656, "fp8_528": 528}


def listed():
    return [
        # one decode step of the two-request, 16-head configuration: the smallest calls, latency alone
        dict(name="append_tiny", op="append", fmt="bf16", b=2, s=1, lo=200, hi=333, ragged=False, style="pairs"),
        # a decode step of 64 requests into the 656-byte cache
        dict(name="append_decode_fp8", op="append", fmt="fp8_656", b=64, s=1, lo=4096, hi=8192, ragged=False, style="pairs"),
        # chunks of a prefill of odd length, padded to the longest, into the 528-byte cache
        dict(name="append_chunk_528", op="append", fmt="fp8_528", b=9, s=1021, lo=1100, hi=9000, ragged=True, style="halves"),
        # a long prompt's chunks into the bf16 cache
        dict(name="append_prefill_bf16", op="append", fmt="bf16", b=16, s=2048, lo=2048, hi=16384, ragged=False, style="pairs"),
        # absorbed queries of a decode step (rotation alone, 576 columns)
        dict(name="query_decode_576", op="query", b=64, s=1, h=128, d=576, norm=False, lo=1024, hi=16384, ragged=False, style="pairs"),
        # heads before absorption (128 + 64 columns), two speculative tokens, normalised
        dict(name="query_spec_192", op="query", b=128, s=2, h=128, d=192, norm=True, lo=1024, hi=16384, ragged=False, style="halves"),
        # 512-wide heads of a prefill chunk with padding, normalised
        dict(name="query_prefill_512", op="query", b=5, s=600, h=64, d=512, norm=True, lo=700, hi=9000, ragged=True, style="pairs"),
        # a decode step of a short-window layer: 64 requests, 128 keys and 4 first tokens each
        dict(name="window_decode_128", op="window", fmt="bf16", b=64, s=1, h=128, window=128, sinks=4, lo=1024, hi=16384, ragged=False, sink_logits=True),
        # two speculative tokens over a long window, 128 heads: the largest
        dict(name="window_spec_4096", op="window", fmt="bf16", b=128, s=2, h=128, window=4096, sinks=64, lo=1024, hi=16384, ragged=False, sink_logits=False),
        # the 656-byte cache, odd window, 64 heads
        dict(name="window_fp8_1000", op="window", fmt="fp8_656", b=48, s=1, h=64, window=1000, sinks=1, lo=500, hi=8192, ragged=False, sink_logits=False),
        # few requests, a long window: work split over the window, 528-byte cache
        dict(name="window_few_528", op="window", fmt="fp8_528", b=3, s=1, h=64, window=8192, sinks=128, lo=8000, hi=32768, ragged=False, sink_logits=False),
        # a chunk of a prompt, 16 heads, padded to the longest
        dict(name="window_prefill_16", op="window", fmt="bf16", b=4, s=333, h=16, window=512, sinks=0, lo=400, hi=4096, ragged=True, sink_logits=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _least(rng, s, most):
    """The shortest length: now and then shorter than the new tokens' slots (a batch padded at its start)."""
    return max(1, s // 2) if rng.random() < 0.1 else s - 1 + _log(rng, 1, most)


def draw(rng):
    op = rng.choice(["append", "query", "window"])
    fmt = rng.choice(["bf16", "fp8_656", "fp8_528"])
    style = rng.choice(["pairs", "halves"])
    ragged = rng.random() < 0.5
    if op == "append":
        s = rng.choice([1, 1, 2, _log(rng, 3, 2048)])
        b = _log(rng, 1, max(1, min(256, 32768 // s)))
        lo = _least(rng, s, 8192)
        return dict(op=op, fmt=fmt, b=b, s=s, lo=lo, hi=lo + _log(rng, 1, 8192), ragged=ragged, style=style)
    if op == "query":
        h = rng.choice([1, 5, 16, 48, 64, 128])
        d = rng.choice([64, 128, 192, 512, 576])
        s = rng.choice([1, 1, 2, _log(rng, 3, 1024)])
        b = _log(rng, 1, max(1, min(256, 100_000_000 // (s * h * d))))
        lo = _least(rng, s, 8192)
        return dict(op=op, b=b, s=s, h=h, d=d, norm=rng.random() < 0.7, lo=lo, hi=lo + _log(rng, 1, 8192), ragged=ragged, style=style)
    h = rng.choice([16, 32, 48, 64, 128])
    window = _log(rng, 1, 8192)
    sinks = rng.choice([0, 1, 4, _log(rng, 1, 256)])
    s = rng.choice([1, 1, 2, _log(rng, 3, 512)])
    b = _log(rng, 1, max(1, min(256, 1_000_000 // (s * (window + sinks)), 300_000 // (s * h))))
    lo = _least(rng, s, 16384)
    return dict(op=op, fmt=fmt, b=b, s=s, h=h, window=window, sinks=sinks, lo=lo, hi=lo + _log(rng, 1, 16384), ragged=ragged,
                sink_logits=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs


def _tokens(case, g, dev):
    """lens [b], new [b] or None, both int32; a request's first page that the step needs, and its page count."""
    lens = torch.randint(case["lo"], case["hi"] + 1, (case["b"],), generator=g, device=dev).int()
    new = torch.randint(1, case["s"] + 1, (case["b"],), generator=g, device=dev).int() if case["ragged"] else None
    return lens, new


def _pages(tokens):
    """Pages that so many tokens in a row touch at most."""
    return (tokens + PAGE - 2) // PAGE + 1


def _block_table(case, lens, first, sink_pages, most, g, dev):
    """Pages in a random order for the page slots that the step reads or writes, -1 elsewhere, and the pool's size:
    ``most`` page slots of a request at most, and one page more that belongs to no request."""
    slots = torch.arange((case["hi"] + PAGE - 1) // PAGE, device=dev)[None]
    live = (slots < ((lens + PAGE - 1) // PAGE)[:, None]) & ((slots < sink_pages) | (slots >= first[:, None]))
    n = case["b"] * most
    pages = torch.randperm(n, generator=g, device=dev).int()
    number = torch.cumsum(live.reshape(-1).int(), 0).reshape(live.shape) - 1
    return torch.where(live, pages[number.clamp(min=0)], -1).int().contiguous(), n + 1


def _rope_table(rows, dev):
    """cos | sin of position * 10000^(-i/32), i = 0 .. 31, in 64 bits, rounded to float32."""
    angle = torch.arange(rows, device=dev, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(32, device=dev, dtype=torch.float64) / 32)
    return torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()


def _encode(x, fmt):
    """float32 rows -> cache rows (bf16, or bytes)."""
    if fmt == "bf16":
        return x.to(torch.bfloat16)
    if fmt == "fp8_656":
        tiles = x[..., :D_LATENT].unflatten(-1, (4, 128))
        amax = tiles.abs().amax(-1)
        scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        codes = (tiles / scale[..., None]).to(torch.float8_e4m3fn).flatten(-2)
        return torch.cat([codes.view(torch.uint8), scale.view(torch.uint8), x[..., D_LATENT:].to(torch.bfloat16).contiguous().view(torch.uint8)], -1)
    blocks = x.unflatten(-1, (16, 32))
    ratio = blocks.abs().amax(-1) / 448.0
    mant, expo = torch.frexp(ratio)  # the smallest power of two at or above the ratio
    expo = torch.where(ratio > 0, torch.where(mant == 0.5, expo - 1, expo), torch.zeros_like(expo)).clamp(-127, 127)
    codes = torch.ldexp(blocks, -expo[..., None]).to(torch.float8_e4m3fn).flatten(-2)
    return torch.cat([codes.view(torch.uint8), (expo + 127).to(torch.uint8)], -1)


def _width(fmt):
    return D_LATENT if fmt == "fp8_528" else D_KEY


def _pool(pages, fmt, g, dev):
    """A cache whose every slot holds some token's row (slots behind a request's length hold what was there before)."""
    rows = torch.randn(pages, PAGE, _width(fmt), generator=g, device=dev)
    return _encode(rows, fmt)


def _inputs(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    lens, new = _tokens(case, g, dev)
    st = dict(case=case, lens=lens, new=new, err=torch.zeros(1, dtype=torch.int32, device=dev))
    count = torch.full_like(lens, case["s"]) if new is None else new
    if case["op"] == "append":
        fmt = case["fmt"]
        st["table"], pages = _block_table(case, lens, (lens - count).clamp(min=0) // PAGE, 0, _pages(case["s"]), g, dev)
        st["cache"] = _pool(pages, fmt, g, dev)
        # the rows come out of a projection beside other columns: a strided view of its output
        wide = torch.randn(case["b"], case["s"], _width(fmt) + 64, generator=g, device=dev).to(torch.bfloat16)
        st["x"] = wide[..., 64:]
        st["weight"] = 1.0 + 0.2 * torch.randn(D_LATENT, generator=g, device=dev)
        st["rope"] = _rope_table(case["hi"], dev)
    elif case["op"] == "query":
        st["q"] = (2.0 * torch.randn(case["b"], case["s"], case["h"], case["d"], generator=g, device=dev)).to(torch.bfloat16)
        st["weight"] = 1.0 + 0.2 * torch.randn(case["d"], generator=g, device=dev) if case["norm"] else None
        st["rope"] = _rope_table(case["hi"], dev)
        st["out"] = torch.zeros_like(st["q"])
    else:
        fmt, w, k = case["fmt"], case["window"], case["sinks"]
        first = (lens - count - w + 1).clamp(min=0) // PAGE
        most = min(_pages(case["s"] + w) + (k + PAGE - 1) // PAGE, (case["hi"] + PAGE - 1) // PAGE)
        st["table"], pages = _block_table(case, lens, first, (k + PAGE - 1) // PAGE, most, g, dev)
        st["cache"] = _pool(pages, fmt, g, dev)
        st["q"] = torch.randn(case["b"], case["s"], case["h"], _width(fmt), generator=g, device=dev).to(torch.bfloat16)
        st["sink_logits"] = torch.randn(case["h"], generator=g, device=dev) if case["sink_logits"] else None
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own and case["op"] == "window":  # the buffers that a serving loop holds for this shape
        from mla_decode_attention_gb300 import binding
        st["buf"] = binding.WindowBuffers(case["b"], case["s"], case["h"], case["window"], case["sinks"], "cuda")
    return st


# ------------------------------------------------------------------ plain forms


def _positions(st):
    """Position of every token slot [b, s] (int64; 0 for padding), and whether it holds a token."""
    lens = st["lens"].long()[:, None]
    count = st["case"]["s"] if st["new"] is None else st["new"].long()[:, None]
    j = torch.arange(st["case"]["s"], device=lens.device)[None]
    pos = lens - count + j
    ok = (j < count) & (pos >= 0)
    return torch.where(ok, pos, torch.zeros_like(pos)), ok


def _rotate(x, cs, style):
    """x [..., 64] by the angles of cs [..., 64] (32 cosines, 32 sines)."""
    c, s = cs[..., :32], cs[..., 32:]
    if style == "pairs":
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    a, b = x[..., :32], x[..., 32:]
    return torch.cat([a * c - b * s, a * s + b * c], -1)


def _rms(x, weight):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight


def _cache_outputs(cache, fmt):
    """What the cache holds: rows, or codes (as e4m3), scales and rotated columns."""
    if fmt == "bf16":
        return (cache,)
    codes = cache[..., :512].view(torch.float8_e4m3fn)
    if fmt == "fp8_656":
        return codes, cache[..., 512:528].view(torch.float32), cache[..., 528:].view(torch.bfloat16)
    return codes, cache[..., 512:].view(torch.float8_e8m0fnu)


def _append_plain(st):
    case, cache = st["case"], st["cache"]
    pos, ok = _positions(st)
    x = st["x"].float()
    cs = st["rope"][pos]
    lat = _rms(x[..., :D_LATENT], st["weight"])
    if case["fmt"] == "fp8_528":
        row = torch.cat([lat[..., :-D_ROPE], _rotate(lat[..., -D_ROPE:], cs, case["style"])], -1)
    else:
        row = torch.cat([lat, _rotate(x[..., D_LATENT:], cs, case["style"])], -1)
    row = _encode(row, case["fmt"])
    page = st["table"].gather(1, pos // PAGE).long()
    spare = cache.shape[0] * PAGE - 1  # padding slots write back what a page of no request holds
    slot = torch.where(ok, page * PAGE + pos % PAGE, spare).reshape(-1)
    flat = cache.view(-1, cache.shape[-1])
    flat[slot] = torch.where(ok.reshape(-1, 1), row.reshape(-1, row.shape[-1]), flat[slot])
    return _cache_outputs(cache, case["fmt"])


def _query_plain(st):
    case = st["case"]
    pos, ok = _positions(st)
    x = st["q"].float()
    if case["norm"]:
        x = _rms(x, st["weight"])
    cs = st["rope"][pos][:, :, None]
    y = torch.cat([x[..., :-D_ROPE], _rotate(x[..., -D_ROPE:], cs, case["style"])], -1).to(torch.bfloat16)
    return torch.where(ok[:, :, None, None], y, st["out"])


def _decode_rows(rows, fmt):
    """Cache rows -> keys in float32: the value is their first 512 columns.  An FP8 key is code * scale rounded to bf16."""
    if fmt == "bf16":
        return rows.float()
    codes = rows[..., :512].contiguous().view(torch.float8_e4m3fn).float()
    if fmt == "fp8_656":
        scale = rows[..., 512:528].contiguous().view(torch.float32)
        rope = rows[..., 528:].contiguous().view(torch.bfloat16).float()
        return torch.cat([(codes.unflatten(-1, (4, 128)) * scale[..., None]).flatten(-2).to(torch.bfloat16).float(), rope], -1)
    scale = torch.exp2(rows[..., 512:].float() - 127.0)
    return (codes.unflatten(-1, (16, 32)) * scale[..., None]).flatten(-2).to(torch.bfloat16).float()


def _visible(st):
    """Key positions [b, s, k] of every token (first tokens, then its window) and whether it sees them."""
    case = st["case"]
    pos, ok = _positions(st)
    pos = pos[..., None]
    w, k = min(case["window"], case["hi"]), min(case["sinks"], case["hi"])
    first = torch.arange(k, device=pos.device)
    last = pos - w + 1 + torch.arange(w, device=pos.device)
    t = torch.cat([first.expand(*pos.shape[:2], k), last], -1)
    seen = torch.cat([(first <= pos - w) & ok[..., None], (last >= 0) & ok[..., None]], -1)
    return t, seen


def _window_plain(st):
    case = st["case"]
    t, seen = _visible(st)
    t = torch.where(seen, t, 0)
    page = st["table"].gather(1, (t // PAGE).flatten(1)).view(t.shape).long().clamp(min=0)
    cache = st["cache"]
    keys = _decode_rows(cache.view(-1, cache.shape[-1])[page * PAGE + t % PAGE], case["fmt"])
    scores = (st["q"].float() * SCALE) @ keys.transpose(-1, -2)
    scores = scores.masked_fill(~seen[:, :, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total))[..., 0]
    out = (p @ keys[..., :D_LATENT]) / torch.where(total > 0, total, torch.ones_like(total))
    if st["sink_logits"] is not None:
        out = out / (1.0 + torch.exp(st["sink_logits"] - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)))[..., None]
    return out.to(torch.bfloat16), lse.transpose(1, 2).contiguous()


# ------------------------------------------------------------------ one pass


def run(state):
    case = state["case"]
    if not own:
        return {"append": _append_plain, "query": _query_plain, "window": _window_plain}[case["op"]](state)
    from mla_decode_attention_gb300 import binding
    formats = {"bf16": binding.MLA_KV_BF16, "fp8_656": binding.MLA_KV_FP8_656, "fp8_528": binding.MLA_KV_FP8_528}
    styles = {"pairs": binding.MLA_ROPE_PAIRS, "halves": binding.MLA_ROPE_HALVES}
    if case["op"] == "append":
        binding.mla_append_kv(state["x"], state["cache"], formats[case["fmt"]], state["table"], state["lens"], rope_table=state["rope"],
                              rope_style=styles[case["style"]], norm_weight=state["weight"], norm_eps=EPS, new_lens=state["new"], err=state["err"])
        return _cache_outputs(state["cache"], case["fmt"])
    if case["op"] == "query":
        binding.mla_query_norm_rope(state["q"], state["out"], state["lens"], rope_table=state["rope"], rope_style=styles[case["style"]],
                                    norm_weight=state["weight"], norm_eps=EPS if case["norm"] else 0.0, new_lens=state["new"], err=state["err"])
        return state["out"]
    buf = state["buf"]
    binding.mla_window_decode(state["q"], state["cache"], formats[case["fmt"]], state["table"], state["lens"], SCALE, case["window"], case["sinks"],
                              buf.num_sm_parts, buf.workspace, buf.out, buf.lse, err=buf.err, attn_sink=state["sink_logits"], new_lens=state["new"])
    return buf.out, buf.lse


# ------------------------------------------------------------------ work and exact values


def work(case):
    tokens = case["b"] * ((case["s"] + 1) / 2 if case["ragged"] else case["s"])
    if case["op"] == "append":
        width = _width(case["fmt"])
        # its columns, its cosines and sines, its cache row; the weights and the table entries once
        return {"bytes": tokens * (2 * width + 4 * 64 + TOKEN_BYTES[case["fmt"]]) + 4 * 512 + 8 * case["b"], "flops": tokens * (4 * 512 + 6 * 32)}
    if case["op"] == "query":
        heads = tokens * case["h"]
        return {"bytes": heads * 4 * case["d"] + tokens * 256 + 4 * case["d"], "flops": heads * (4 * case["d"] * case["norm"] + 6 * 32)}
    mean = (case["lo"] + case["hi"]) / 2
    per = tokens / case["b"]
    keys = min(mean, case["window"] + case["sinks"])
    union = min(mean, case["window"] + case["sinks"] + per - 1)
    width = _width(case["fmt"])
    rows = tokens * case["h"]
    return {"bytes": case["b"] * union * TOKEN_BYTES[case["fmt"]] + rows * (2 * width + 2 * 512 + 4), "flops": 2 * rows * keys * (width + 512)}


def _keys_by_bits(rows, fmt):
    """Keys in 64 bits from the formats' definitions: e4m3 is sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    if fmt == "bf16":
        return rows.double()
    code = torch.arange(256, device=rows.device)
    sign, e, m = 1.0 - 2.0 * (code // 128).double(), (code // 8 % 16).double(), (code % 8).double()
    value = sign * torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.pow(2.0, e - 7))
    value = value[rows[:, :512].long()]
    if fmt == "fp8_656":
        scale = rows[:, 512:528].contiguous().view(torch.float32).double().repeat_interleave(128, -1)
        return torch.cat([(value * scale).to(torch.bfloat16), rows[:, 528:].contiguous().view(torch.bfloat16)], -1).double()
    return value * torch.pow(2.0, rows[:, 512:].double() - 127).repeat_interleave(32, -1)


def exact(case, seed):
    """The definitions in 64 bits, one token and request after another in arrays of their own."""
    st = _inputs(case, seed)
    dev = st["lens"].device
    lens = st["lens"].double()
    count = st["new"].double() if st["new"] is not None else torch.full_like(lens, case["s"])
    slot = torch.arange(case["s"], device=dev, dtype=torch.float64).repeat(case["b"], 1)
    where = (lens - count)[:, None] + slot
    real = (slot < count[:, None]) & (where >= 0)
    where = where.long()
    if case["op"] in ("append", "query"):
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=dev),
                           where[..., None].double() / torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=dev), torch.arange(32, device=dev, dtype=torch.float64) / 32))

        def turned(x, by):
            z = torch.complex(*(x.unflatten(-1, (32, 2)).unbind(-1) if case["style"] == "pairs" else x.unflatten(-1, (2, 32)).unbind(-2))) * by
            return torch.stack([z.real, z.imag], -1 if case["style"] == "pairs" else -2).flatten(-2)

        if case["op"] == "query":
            x = st["q"].double()
            if case["norm"]:
                x = x / ((x.square().sum(-1, keepdim=True) / case["d"] + EPS).sqrt()) * st["weight"].double()
            x[..., case["d"] - 64:] = turned(x[..., case["d"] - 64:], turn[:, :, None])
            return torch.where(real[..., None, None], x, torch.zeros_like(x))
        x = st["x"].double()
        x[..., :512] = x[..., :512] / (x[..., :512].square().sum(-1, keepdim=True) / 512 + EPS).sqrt() * st["weight"].double()
        x[..., -64:] = turned(x[..., -64:], turn)
        x = x[real]
        request = torch.arange(case["b"], device=dev)[:, None].expand_as(where)[real]
        page, offset = st["table"].long()[request, where[real] // 64], where[real] % 64
        held = [v.double() if v.dtype != torch.float8_e8m0fnu else torch.pow(2.0, v.contiguous().view(torch.uint8).double() - 127) for v in _cache_outputs(st["cache"], case["fmt"])]
        if case["fmt"] == "bf16":
            held[0][page, offset] = x
        elif case["fmt"] == "fp8_656":
            scale = x[:, :512].unflatten(-1, (4, 128)).abs().max(-1).values / 448
            held[0][page, offset] = x[:, :512] / scale.repeat_interleave(128, -1)
            held[1][page, offset] = scale
            held[2][page, offset] = x[:, 512:]
        else:
            scale = torch.pow(2.0, torch.ceil(torch.log2(x.unflatten(-1, (16, 32)).abs().max(-1).values / 448)))
            held[0][page, offset] = x / scale.repeat_interleave(32, -1)
            held[1][page, offset] = scale
        return tuple(held)
    if case["b"] * case["s"] * case["h"] * min(case["window"] + case["sinks"], case["hi"]) * 2 * (_width(case["fmt"]) + 512) > 4e11:
        return None  # over the time that this function may take
    out = torch.zeros(case["b"], case["s"], case["h"], 512, dtype=torch.float64, device=dev)
    lse = torch.full((case["b"], case["h"], case["s"]), -math.inf, dtype=torch.float64, device=dev)
    lengths, tables = st["lens"].tolist(), st["table"].long().clamp(min=0)
    per = 64  # tokens of a request at a time
    for b in range(case["b"]):
        at = torch.arange(lengths[b], device=dev)
        for j in range(0, case["s"], per):
            here = where[b, j:j + per]
            low = max(0, int(here.min()) - case["window"] + 1)
            use = at[(at < case["sinks"]) | (at >= low)]
            if not len(use):
                continue
            k = _keys_by_bits(st["cache"][tables[b, use // 64], use % 64], case["fmt"])
            sees = (use <= here[:, None]) & ((use < case["sinks"]) | (use > here[:, None] - case["window"])) & real[b, j:j + per, None]
            score = torch.einsum("shd,kd->shk", st["q"][b, j:j + per].double(), k) * SCALE
            score[~sees[:, None].expand_as(score)] = -math.inf
            total = torch.logsumexp(score, -1)
            weight = torch.where(torch.isinf(total)[..., None], torch.zeros_like(score), torch.exp(score - total[..., None]))
            value = torch.einsum("shk,kd->shd", weight, k[:, :512])
            if st["sink_logits"] is not None:
                value = value * torch.sigmoid(total - st["sink_logits"].double())[..., None]
            out[b, j:j + per], lse[b, :, j:j + per] = value, total.T
    return out, lse
