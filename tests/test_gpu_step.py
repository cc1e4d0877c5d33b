"""A layer's step as it is run: append, query, windowed and dense attention on
one cache, on a stream of its own, captured into a graph and replayed while the
lengths grow."""
import numpy as np
import pytest
import torch

import oracle
from mla_decode_attention_gb300 import binding, workloads
from tests._util import assert_parity_per_token, f64_np
from tests.test_gpu_append import DEV, library, rope_table  # noqa: F401
from tests.test_gpu_window import keys_of

pytestmark = pytest.mark.gpu

FORMATS = [binding.MLA_KV_BF16, binding.MLA_KV_FP8_656, binding.MLA_KV_FP8_528]
WINDOW, SINKS, SCALE = 90, 3, workloads.SOFTMAX_SCALE


class Layer:
    def __init__(self, fmt, b, s, h, most, seed):
        g = torch.Generator().manual_seed(seed)
        self.fmt, self.b, self.s, self.h = fmt, b, s, h
        self.d = 512 if fmt == FORMATS[2] else 576
        slots = (most + 63) // 64
        self.table = torch.randperm(b * slots, generator=g).view(b, slots).int().to(DEV)
        shape = (b * slots, 64, {FORMATS[0]: 576, FORMATS[1]: 656, FORMATS[2]: 528}[fmt])
        self.cache = torch.zeros(shape, dtype=torch.bfloat16 if fmt == FORMATS[0] else torch.uint8, device=DEV)
        self.rope = rope_table(most).to(DEV)
        self.w = (1 + 0.2 * torch.randn(512, generator=g)).to(DEV)
        self.lens = torch.zeros(b, dtype=torch.int32, device=DEV)
        self.x = torch.zeros(b, s, self.d, dtype=torch.bfloat16, device=DEV)
        self.q = torch.zeros(b, s, h, self.d, dtype=torch.bfloat16, device=DEV)
        self.win = binding.WindowBuffers(b, s, h, WINDOW, SINKS, DEV)
        self.dense = binding.DecodeBuffers(b, s, h, DEV)

    def step(self):
        binding.mla_append_kv(self.x, self.cache, self.fmt, self.table, self.lens, self.rope, 0, self.w, 1e-6, None, self.win.err)
        binding.mla_query_norm_rope(self.q, self.q, self.lens, self.rope, 0, None, 1e-6, None, self.win.err)
        binding.mla_window_decode(self.q, self.cache, self.fmt, self.table, self.lens, SCALE, WINDOW, SINKS, self.win.num_sm_parts,
                                  self.win.workspace, self.win.out, self.win.lse, self.win.err)
        d = self.dense
        binding.mla_get_metadata(self.lens, self.b, self.s, True, 0, d.num_sm_parts, d.metadata)
        binding.mla_decode(self.q, self.cache, self.fmt, self.table, self.lens, SCALE, True, d.metadata, d.num_sm_parts, d.workspace,
                           d.out, d.lse, d.err)

    def load(self, g, grow):
        """New inputs for the next step: every request grows by s tokens."""
        self.x.copy_(torch.randn(self.x.shape, generator=g).to(torch.bfloat16))
        q = torch.randn(self.q.shape, generator=g).to(torch.bfloat16)
        self.q.copy_(q)
        self.lens += grow
        return self.x.cpu(), q


def check(layer, plain, q):
    """The step's outputs against the oracle: keys from what the cache holds
    (checked against the plain rows), queries from the oracle's rotation."""
    lens = layer.lens.cpu().tolist()
    keys = keys_of(layer.cache.cpu(), layer.fmt)
    table = layer.table.cpu().numpy()
    rope, w = f64_np(layer.rope), f64_np(layer.w)
    for b, L in enumerate(lens):
        rows = np.concatenate([x[b] for x in plain])      # every token appended so far
        at = np.arange(L)
        want = oracle.latent_rows(rows, at, rope, False, w, 1e-6, layer.d == 512)
        got = keys[table[b, at // 64], at % 64]
        # coarsest format: e4m3 half step 2^-4, its bf16 value half a step more
        step = 2.0 ** -8 if layer.fmt == FORMATS[0] else 2.0 ** -4 + 2.0 ** -8
        top = np.abs(want[:, :512]).max(-1, keepdims=True)
        assert np.all(np.abs(got - want) <= step * np.abs(want) * 1.001 + 2.0 ** -10 * top / 224 + 2.0 ** -15 * 4)
    pos = oracle.token_positions(lens, None, layer.s)
    qr = oracle.query_rows(f64_np(q).reshape(-1, layer.h, layer.d), pos.reshape(-1), rope, False, None, 1e-6).reshape(q.shape)
    qb = f64_np(layer.q)
    assert np.all(np.abs(qb - qr) <= 2.0 ** -8 * np.abs(qr) + 2.0 ** -15 * 4)
    # attention from the queries and keys that the step itself left (their rounding is checked above)
    o, l = oracle.window_decode(qb, keys, table, lens, None, SCALE, WINDOW, SINKS)
    assert_parity_per_token(f64_np(layer.win.out), o, f64_np(layer.win.lse), l, "window")
    o, l = oracle.window_decode(qb, keys, table, lens, None, SCALE, 2**31 - 1, 0)
    assert_parity_per_token(f64_np(layer.dense.out), o, f64_np(layer.dense.lse), l, "dense")
    assert int(layer.win.err.item()) == 0 and int(layer.dense.err.item()) == 0


@pytest.mark.parametrize("fmt,h", [(FORMATS[0], 128), (FORMATS[0], 16), (FORMATS[1], 64), (FORMATS[2], 128)])
def test_prompt_then_tokens(fmt, h):
    g = torch.Generator().manual_seed(1)
    layer = Layer(fmt, 2, 5, h, 200, 2)
    plain = []
    for _ in range(30):
        x, q = layer.load(g, layer.s)
        plain.append(f64_np(x))
        layer.step()
    torch.cuda.synchronize()
    check(layer, plain, q)


@pytest.mark.parametrize("fmt,h", [(FORMATS[0], 128), (FORMATS[1], 48)])
def test_captured_step_is_replayed_while_lengths_grow(fmt, h):
    g = torch.Generator().manual_seed(3)
    layer = Layer(fmt, 3, 1, h, 260, 4)
    stream = torch.cuda.Stream()
    plain = []
    x, q = layer.load(g, 1)
    plain.append(f64_np(x))
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        layer.step()                                    # warm-up on the stream: kernel attributes are set
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    layer.q.copy_(q)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        layer.step()
    for _ in range(240):
        x, q = layer.load(g, 1)
        plain.append(f64_np(x))
        graph.replay()
        torch.cuda.synchronize()
    check(layer, plain, q)


def test_two_layers_on_two_streams():
    """Two layers with buffers of their own run at once."""
    layers = [Layer(FORMATS[0], 2, 2, 128, 300, 5), Layer(FORMATS[0], 2, 2, 64, 300, 6)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    gens = [torch.Generator().manual_seed(7), torch.Generator().manual_seed(8)]
    plain = [[], []]
    last = [None, None]
    for _ in range(60):
        for i in (0, 1):
            x, last[i] = layers[i].load(gens[i], 2)
            plain[i].append(f64_np(x))
        torch.cuda.synchronize()
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                layers[i].step()
        torch.cuda.synchronize()
    for i in (0, 1):
        check(layers[i], plain[i], last[i])


def test_stream_argument_is_the_one_used():
    layer = Layer(FORMATS[0], 2, 1, 16, 100, 9)
    x, q = layer.load(torch.Generator().manual_seed(10), 1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()                      # whatever is launched elsewhere breaks the capture
    with torch.cuda.graph(graph, stream=s):
        binding.mla_append_kv(layer.x, layer.cache, layer.fmt, layer.table, layer.lens, layer.rope, 0, layer.w, 1e-6, stream=s)
        binding.mla_query_norm_rope(layer.q, layer.q, layer.lens, layer.rope, stream=s.cuda_stream)
    assert float(layer.cache.float().abs().sum()) == 0
    graph.replay()
    torch.cuda.synchronize()
    assert float(layer.cache.float().abs().sum()) > 0
