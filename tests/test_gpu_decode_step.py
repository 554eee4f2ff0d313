"""GPU: a layer's attention side as a serving program runs it -- qkv product,
rotary, cache write, attention, output product -- for a prompt and several
decode steps, each stage checked against the oracle on what the GPU handed
it; captured graphs, streams and workspaces."""
import numpy as np
import pytest
import torch

import oracle
import quantized_gemm_packed_amd as hum
import synth
from gpu_util import assert_tol, bf16_bits_of, descs, dev, f64, prepare
from test_gpu_kv import Case
from test_gpu_rotary import _check as check_rotary

pytestmark = pytest.mark.gpu


class Layer:
    """hidden 256, 4 query and 2 key-value heads of 64, UINT4 weights."""
    hid, hq, hk, d, ps = 256, 4, 2, 64, 16

    def __init__(self, fmt, pages):
        n = (self.hq + 2 * self.hk) * self.d
        self.wqkv = synth.dense_w4a16(9001, 1, n, self.hid, group=128, asym=True)
        self.wo = synth.dense_w4a16(9002, 1, self.hid, self.hq * self.d, group=128, asym=True)
        self.dq, self.oq = descs("uint4", "group", 128, "bf16", 1, n, self.hid, zero=True)
        self.do, self.oo = descs("uint4", "group", 128, "bf16", 1, self.hid, self.hq * self.d, zero=True)
        self.pq, self.po = prepare(self.dq, self.wqkv, "bf16"), prepare(self.do, self.wo, "bf16")
        self.kv = hum.make_kv_desc(fmt, pages, self.ps, self.hk, self.d)
        self.cache = torch.zeros(hum.kv_cache_bytes(self.kv), dtype=torch.uint8, device="cuda")
        f, self.factor = hum.rotary_inv_freq(self.d, scaling="yarn", factor=4.0, original_len=1024)
        self.freq = f.cuda()

    def append(self, x, pos, slots):
        """Positions and cache of new tokens -> their rotated queries."""
        qkv = hum.linear(self.dq, self.pq, x).view(-1, self.hq + 2 * self.hk, self.d)
        q, k, v = qkv.split([self.hq, self.hk, self.hk], 1)
        qr, kr = hum.rotary(q, k, pos, self.freq, factor=self.factor)
        hum.kv_write(self.kv, self.cache, kr, v, slots)
        return qkv, qr, kr, v

    def step(self, x, pos, slots, table, lens, **kw):
        qkv, qr, kr, v = self.append(x, pos, slots)
        att = hum.kv_attention(self.kv, self.cache, qr, table, lens, **kw)
        out = hum.linear(self.do, self.po, att.view(-1, self.hq * self.d))
        return qkv, qr, kr, v, att, out


def _x(seed, t, hid):
    return dev(synth.bf16_normal(synth.rng(seed), (t, hid)))


@pytest.mark.parametrize("fmt", ["bf16", "fp8_token", "mxfp8", "mxfp4"])
def test_prompt_and_decode_steps(fmt):
    ly = Layer(fmt, 40)
    lens = np.array([37, 1, 100])
    per = 10
    table = np.random.default_rng(1).permutation(40)[:3 * per].reshape(3, per).astype(np.int32)
    ref = oracle.attention.Cache(fmt, 40, ly.ps, ly.hk, ly.d)
    seq = np.repeat(np.arange(3), lens)
    pos = np.concatenate([np.arange(n) for n in lens])

    def slots_of(seq, pos):
        return table[seq, pos // ly.ps].astype(np.int64) * ly.ps + pos % ly.ps

    _, _, kr, v = ly.append(_x(70, len(pos), ly.hid), dev(pos), dev(slots_of(seq, pos)))
    ref.write(slots_of(seq, pos), bf16_bits_of(kr), bf16_bits_of(v))
    assert np.array_equal(ly.cache.cpu().numpy(), ref.buf.reshape(-1))
    c = Case.__new__(Case)                 # its tolerance, on this cache
    c.cache, c.table, c.d = ref, table, ly.d
    for s in range(3):
        pos, seq = lens.copy(), np.arange(3)
        lens = lens + 1
        slots = slots_of(seq, pos)
        x = _x(80 + s, 3, ly.hid)
        qkv, qr, kr, v, att, out = ly.step(x, dev(pos), dev(slots), dev(table), dev(lens.astype(np.int32)),
                                           return_lse=False)
        assert_tol(qkv.flatten(1), oracle.gemm.linear(ly.oq, f64(x), ly.wqkv["codes"], ly.wqkv["scales"],
                                                      ly.wqkv["zeros"]), "qkv")
        for y, z in ((qr, qkv[:, :ly.hq]), (kr, qkv[:, ly.hq:ly.hq + ly.hk])):
            check_rotary(y, z, pos, ly.freq.cpu().numpy(), "half", np.float32(ly.factor), False, "rotary")
        ref.write(slots, bf16_bits_of(kr), bf16_bits_of(v))
        assert np.array_equal(ly.cache.cpu().numpy(), ref.buf.reshape(-1))
        c.q, c.lens = f64(qr), lens
        got = hum.kv_attention(ly.kv, ly.cache, qr, dev(table), dev(lens.astype(np.int32)), return_lse=True)
        assert torch.equal(got[0], att)
        c.check(got, what=f"step {s}")
        assert_tol(out, oracle.gemm.linear(ly.oo, f64(att).reshape(3, -1), ly.wo["codes"], ly.wo["scales"],
                                           ly.wo["zeros"]), "output")


def test_captured_step_replays_with_growing_sequences():
    """One captured step, replayed while its inputs (tokens, positions, slots,
    lengths) change in place, against eager steps on a second cache."""
    ly, eager = Layer("mxfp8", 40), Layer("mxfp8", 40)
    table = torch.arange(30, dtype=torch.int32, device="cuda").view(2, 15)
    x = torch.zeros((2, ly.hid), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(2, dtype=torch.int64, device="cuda")
    slots, lens = torch.zeros_like(pos), torch.zeros(2, dtype=torch.int32, device="cuda")

    def feed(s, n0):
        x.copy_(_x(300 + s, 2, ly.hid))
        pos.copy_(torch.tensor(n0))
        slots.copy_(table.gather(1, (pos // ly.ps)[:, None]).squeeze(1).long() * ly.ps + pos % ly.ps)
        lens.copy_(pos + 1)

    feed(0, [0, 0])
    for _ in range(2):
        ly.step(x, pos, slots, table, lens)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = ly.step(x, pos, slots, table, lens)
    for s in range(40):
        feed(s, [s, s * 5])
        want = eager.step(x, pos, slots, table, lens)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(res, want):
            assert torch.equal(a, b), s
    assert torch.equal(ly.cache, eager.cache)


def test_two_graphs_of_one_capture_stream_replayed_on_two_streams():
    """Each captured attention has scratch of its own: replays of two graphs
    that overlap in time leave each other's parts alone."""
    cases = [Case(50 + i, "bf16", [9000, 700], 8, 1, 64, 64) for i in range(2)]
    want = [c.run(return_lse=True) for c in cases]
    torch.cuda.synchronize()
    graphs, got = [], []
    cap = torch.cuda.Stream()
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=cap):
            got.append(c.run(return_lse=True))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_side_streams_and_shared_workspaces():
    """Calls on two streams at once (the binding's scratch is per stream), and
    one caller workspace used by the attention and a Stream-K product in
    turn (both leave its header zero)."""
    a, b = (Case(60 + i, f, [5000, 300, 20], 8, 2, 128, 32) for i, f in enumerate(("fp8_token", "mxfp4")))
    wa, wb = a.run(), b.run()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(sa):
            ra = a.run()
        with torch.cuda.stream(sb):
            rb = b.run()
    torch.cuda.synchronize()
    assert torch.equal(ra, wa) and torch.equal(rb, wb)
    n, k, m = 640, 2048, 32
    case = synth.dense_w4a16(synth.seed_for(9, m), m, n, k, group=128, asym=True)
    hd, _ = descs("uint4", "group", 128, "bf16", 1, n, k, zero=True)
    packed, x = prepare(hd, case, "bf16"), dev(case["x"])
    lin = hum.linear(hd, packed, x)
    nb = max(hum.linear_workspace_bytes(hd, m), hum.kv_attention_workspace_bytes(a.desc, 8, 3, a.table.shape[1]))
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(a.run(workspace=ws), wa)
        assert torch.equal(hum.linear(hd, packed, x, workspace=ws), lin)
    assert not ws[:64 << 10].any()


def test_attention_table_of_millions_of_pages():
    """A block table as wide as the longest sequences a call may have, its
    entries past the lengths never read as pages."""
    c = Case(70, "bf16", [3000, 0, 129], 4, 2, 64, 16)
    mp = 6_000_000
    wide = torch.full((3, mp), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.dev["block_table"]
    got, want = c.run(return_lse=True, block_table=wide), c.run(return_lse=True)
    c.check(got, what="wide")
    # the narrow table's call may run on fewer workgroups, the bits then differ; the values hold either way
    c.check(want, what="narrow")


def test_attention_thousands_of_sequences():
    g = np.random.default_rng(71)
    lens = [int(n) for n in g.integers(0, 4, 5000)]
    lens[4999], lens[100] = 700, 300
    c = Case(72, "bf16", lens, 1, 1, 64, 16)
    c.check(c.run(return_lse=True), what="thousands")
