"""A prompt as it is run: its rows appended, read back, projected up, attended in one piece or in several that are
merged; against the absorbed form of the same attention over the same cache, on streams and in captured graphs."""
import numpy as np
import pytest
import torch

import oracle
from mla_decode_attention_gb300 import binding
from tests._util import LSE_ABS, f64_np
from tests.test_gpu_append import DEV, FORMATS, library, rope_table  # noqa: F401
from tests.test_gpu_prefill import case, check, definition
from tests.test_gpu_window import keys_of

pytestmark = pytest.mark.gpu

H, SCALE = 16, 192 ** -0.5


class Layer:
    """Requests with a cached context and a chunk of new tokens each."""

    def __init__(self, fmt, ctx, new, seed, slots=None):
        g = torch.Generator().manual_seed(seed)
        make = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.fmt, self.b, self.ctx, self.new = fmt, len(ctx), ctx, new
        lens = [c + n for c, n in zip(ctx, new)]
        slots = slots or (max(lens) + 63) // 64
        self.table = torch.randperm(self.b * slots, generator=g).view(self.b, slots).int().to(DEV)
        wide = {FORMATS[0]: 576, FORMATS[1]: 656}[fmt]
        self.cache = torch.zeros(self.b * slots, 64, wide, dtype=torch.bfloat16 if fmt == FORMATS[0] else torch.uint8, device=DEV)
        self.rope = rope_table(max(lens)).to(DEV)
        self.up = (make(H * 256, 512) / 512 ** 0.5).to(torch.bfloat16).to(DEV)      # per head: 128 rows of W_k, 128 of W_v
        self.lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        most = max(lens)
        x = torch.zeros(self.b, most, 576)
        for i, n in enumerate(lens):
            x[i, :n] = make(n, 576)
        self.x = x.to(torch.bfloat16).to(DEV)
        binding.mla_append_kv(self.x, self.cache, fmt, self.table, self.lens, self.rope, 0, None, 1e-6, self.lens)
        starts = lambda n: torch.tensor([0] + np.cumsum(n).tolist(), dtype=torch.int32, device=DEV)  # noqa: E731
        self.cu_q, self.cu_k, self.cu_c = starts(new), starts(lens), starts(ctx)
        self.q = make(sum(new), H, 192).to(torch.bfloat16).to(DEV)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.ctx_starts = torch.tensor(ctx, dtype=torch.int32, device=DEV)
        self.rows_all = torch.zeros(sum(lens), 576, dtype=torch.bfloat16, device=DEV)
        self.buf = binding.PrefillBuffers(sum(new), sum(lens), self.b, H, H, DEV)
        # in two pieces: the context (all of it seen), the chunk itself (causal)
        self.rows = [torch.zeros(sum(n), 576, dtype=torch.bfloat16, device=DEV) for n in (ctx, new)]
        self.piece = [binding.PrefillBuffers(sum(new), sum(n), self.b, H, H, DEV) for n in (ctx, new)]
        self.parts = torch.zeros(2, sum(new), H, 128, dtype=torch.bfloat16, device=DEV)
        self.lses = torch.zeros(2, H, sum(new), device=DEV)
        self.out, self.lse = torch.zeros_like(self.parts[0]), torch.zeros_like(self.lses[0])

    def project(self, rows):
        both = (rows[:, :512] @ self.up.T).view(-1, H, 256)
        return both[..., :128], both[..., 128:]

    def whole(self):
        binding.mla_gather_kv(self.cache, self.fmt, self.table, self.cu_k, self.rows_all, None, self.err)
        k, v = self.project(self.rows_all)
        b = self.buf
        binding.mla_prefill(self.q, k, v, self.cu_q, self.cu_k, SCALE, True, b.num_sm_parts, b.workspace, b.out, b.lse,
                            self.rows_all[:, 512:], self.err)

    def pieces(self):
        for i, (cu, first, causal) in enumerate(((self.cu_c, None, False), (self.cu_q, self.ctx_starts, True))):
            binding.mla_gather_kv(self.cache, self.fmt, self.table, cu, self.rows[i], first, self.err)
            k, v = self.project(self.rows[i])
            b = self.piece[i]
            binding.mla_prefill(self.q, k, v, self.cu_q, cu, SCALE, causal, b.num_sm_parts, b.workspace, self.parts[i], self.lses[i],
                                self.rows[i][:, 512:], self.err)
        binding.mla_merge_states(self.parts, self.lses, self.out, self.lse)

    def wanted(self):
        """The absorbed form in 64 bits over what the cache holds.  Keys and values projected up are rounded to bf16 on
        the way here, which the absorbed form does not do."""
        keys = keys_of(self.cache.cpu(), self.fmt)
        w = f64_np(self.up).reshape(H, 2, 128, 512)
        q, table = f64_np(self.q), self.table.cpu().numpy()
        out, lse = [], []
        at = 0
        for i in range(self.b):
            for j in range(self.new[i]):
                t = np.arange(self.ctx[i] + j + 1)
                rows = np.concatenate([np.einsum("hd,hdc->hc", q[at, :, :128], w[:, 0]), q[at, :, 128:]], 1)
                o, l = oracle.attend(rows, keys[table[i, t // 64], t % 64], SCALE)
                out.append(np.einsum("hc,hdc->hd", o, w[:, 1]))
                lse.append(l)
                at += 1
        return np.stack(out), np.stack(lse, 1)


def near(out, lse, want, want_lse):
    """Rounded keys, values, weights and outputs: four independent roundings to bf16 (2^-8 each at most, a third of its
    square on average): rel-L2 below 4 * 2^-8 / sqrt(3) = 9e-3; a score of size s moves by 2^-8 of sum |q k| over its
    128 rounded columns at most, at random by a tenth of that."""
    o, l = f64_np(out), f64_np(lse)
    assert np.linalg.norm(o - want) <= 9e-3 * np.linalg.norm(want)
    assert np.max(np.abs(l - want_lse)) <= 2e-2


@pytest.mark.parametrize("fmt", FORMATS[:2])
@pytest.mark.parametrize("ctx,new", [([0, 0], [200, 65]), ([300, 0, 1000], [40, 130, 1]), ([64, 640], [64, 1])])
def test_prompt(fmt, ctx, new):
    layer = Layer(fmt, ctx, new, len(ctx))
    layer.whole()
    layer.pieces()
    torch.cuda.synchronize()
    assert int(layer.err.item()) == 0
    want, want_lse = layer.wanted()
    near(layer.buf.out, layer.buf.lse, want, want_lse)
    near(layer.out, layer.lse, want, want_lse)
    # the same keys in one piece and in two: parts rounded to bf16 once more
    a, b = f64_np(layer.buf.out), f64_np(layer.out)
    assert np.linalg.norm(a - b) <= 4e-3 * np.linalg.norm(a)
    assert np.max(np.abs(f64_np(layer.buf.lse) - f64_np(layer.lse))) <= LSE_ABS


def test_captured_and_replayed_with_other_lengths():
    """The calls of one capture serve whatever lengths and pages the tensors hold when it is replayed."""
    layer = Layer(FORMATS[1], [300, 500], [64, 64], 5, slots=10)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        layer.whole()
        layer.pieces()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        layer.whole()
        layer.pieces()
    for ctx, new in (([500, 300], [64, 64]), ([300, 500], [1, 127]), ([300, 500], [64, 64])):
        other = Layer(FORMATS[1], ctx, new, 6, slots=10)
        for name in ("table", "cache", "cu_q", "cu_k", "cu_c", "q", "ctx_starts", "up"):
            getattr(layer, name).copy_(getattr(other, name))
        layer.ctx, layer.new = ctx, new
        graph.replay()
        torch.cuda.synchronize()
        want, want_lse = layer.wanted()
        near(layer.buf.out, layer.buf.lse, want, want_lse)
        near(layer.out, layer.lse, want, want_lse)
    assert int(layer.err.item()) == 0


def test_two_streams_at_once():
    layers = [Layer(FORMATS[0], [400, 0], [30, 200], 7), Layer(FORMATS[1], [10, 900], [100, 20], 8)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for layer, s in zip(layers, streams):
            with torch.cuda.stream(s):
                layer.whole()
                layer.pieces()
    torch.cuda.synchronize()
    for layer in layers:
        want, want_lse = layer.wanted()
        near(layer.buf.out, layer.buf.lse, want, want_lse)
        near(layer.out, layer.lse, want, want_lse)


def test_stream_argument_is_the_one_used():
    layer = Layer(FORMATS[0], [100], [20], 9)
    layer.whole()
    k, v = layer.project(layer.rows_all)
    torch.cuda.synchronize()
    layer.rows_all.zero_()
    layer.buf.out.zero_()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        binding.mla_gather_kv(layer.cache, layer.fmt, layer.table, layer.cu_k, layer.rows_all, stream=s)
        binding.mla_prefill(layer.q, k, v, layer.cu_q, layer.cu_k, SCALE, True, 152, layer.buf.workspace, layer.buf.out, layer.buf.lse,
                            layer.rows_all[:, 512:], stream=s.cuda_stream)
        binding.mla_merge_states(layer.parts[:1], layer.lses[:1], layer.out, layer.lse, s)
    torch.cuda.synchronize()
    assert float(layer.rows_all.float().abs().sum()) == 0 and float(layer.buf.out.float().abs().sum()) == 0
    graph.replay()
    torch.cuda.synchronize()
    assert float(layer.buf.out.float().abs().sum()) > 0


def test_calls_one_after_the_other_see_each_other():
    """A call's outputs are the next one's queries and values, without anything between them."""
    c = case([300, 77], [300, 77], 4, rope="none")
    q, k, v = (c[n].contiguous().to(DEV) for n in ("q", "k", "v"))
    cu = torch.tensor(c["cu_q"], dtype=torch.int32, device=DEV)
    bufs = [binding.PrefillBuffers(377, 377, 2, 4, 4, DEV) for _ in range(6)]
    for _ in range(3):
        a, b = q, v
        for buf in bufs:
            binding.mla_prefill(a, k, b, cu, cu, c["scale"], True, buf.num_sm_parts, buf.workspace, buf.out, buf.lse, None, buf.err)
            a, b = buf.out, buf.out
    torch.cuda.synchronize()
    a, b = q, v
    for buf in bufs:
        d = dict(c, q=a.cpu(), v=b.cpu(), err=int(buf.err.item()))
        check(d, buf.out.cpu(), buf.lse.cpu())
        a, b = buf.out, buf.out
