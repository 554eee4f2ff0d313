"""GPU: a whole MoE decoder layer from the library's calls alone -- norm with
quantized output, qkv product, head norms with rotary and the cache's append,
attention, output product, residual and norm, router product, routing, expert
layer -- for a prompt and decode steps, every stage checked against the oracle
on what the GPU handed it; captured graphs and streams."""
import numpy as np
import pytest
import torch

import oracle
import quantized_gemm_packed_amd as hum
import synth
from gpu_util import assert_tol, bf16_bits_of, descs, dev, f64, prepare
from test_gpu_kv import Case as Attention
from test_gpu_rms_norm import EPS, _near, check_codes
from test_gpu_rotary_kv_write import Case as Append

pytestmark = pytest.mark.gpu
L = oracle.layer


class Layer:
    """hidden 256, 4 query and 2 key-value heads of 64 with head norms, 8 experts of 128, the best 2 of 2 of 4 groups."""
    hid, hq, hk, d, ps, experts, inter, topk = 256, 4, 2, 64, 16, 8, 128, 2
    routing = dict(score="sigmoid", num_groups=4, topk_groups=2, group_score="top2", scale=1.5)

    def __init__(self, fmt, pages):
        n = (self.hq + 2 * self.hk) * self.d
        g = torch.Generator().manual_seed(7)
        bf = lambda *s: (1 + 0.1 * torch.randn(*s, generator=g)).to(torch.bfloat16).cuda()  # noqa: E731
        self.w_in, self.w_post, self.w_q, self.w_k = bf(self.hid), bf(self.hid), bf(self.d), bf(self.d)
        self.bias = 0.05 * torch.randn(self.experts, generator=g).cuda()
        self.wqkv = synth.quant_weights(9101, "e4m3", "channel", 0, "f32", 1, n, self.hid)
        self.dq, self.oq = descs("e4m3", "channel", 0, "f32", 1, n, self.hid, act="fp8_token")
        self.pq = prepare(self.dq, self.wqkv, "f32")
        self.wo = synth.dense_w4a16(9102, 1, self.hid, self.hq * self.d, group=128, asym=True)
        self.do, self.oo = descs("uint4", "group", 128, "bf16", 1, self.hid, self.hq * self.d, zero=True)
        self.po = prepare(self.do, self.wo, "bf16")
        self.wr = synth.quant_weights(9103, "int8", "channel", 0, "f32", 1, self.experts, self.hid)
        self.dr, self.our = descs("int8", "channel", 0, "f32", 1, self.experts, self.hid)
        self.pr = prepare(self.dr, self.wr, "f32")
        self.w13 = synth.moe_weights_mxfp4(9104, self.experts, 2 * self.inter, self.hid)
        self.w2 = synth.moe_weights_mxfp4(9105, self.experts, self.hid, self.inter)
        self.d13, self.o13 = descs("e2m1", "group", 32, "e8m0", self.experts, 2 * self.inter, self.hid)
        self.d2, self.o2 = descs("e2m1", "group", 32, "e8m0", self.experts, self.hid, self.inter)
        self.p13, self.p2 = prepare(self.d13, self.w13, "e8m0"), prepare(self.d2, self.w2, "e8m0")
        self.kv = hum.make_kv_desc(fmt, pages, self.ps, self.hk, self.d)
        self.cache = torch.full((hum.kv_cache_bytes(self.kv),), 0xA5, dtype=torch.uint8, device="cuda")
        f, self.factor = hum.rotary_inv_freq(self.d, scaling="yarn", factor=4.0, original_len=1024)
        self.freq = f.cuda()

    def append(self, x, stream, pos, slots):
        """Everything before the attention -> what each stage gave."""
        (a, a_s), stream = hum.rms_norm(x, self.w_in, residual=stream, act_fmt="fp8_token")
        qkv = hum.linear(self.dq, self.pq, a, a_scales=a_s).view(-1, self.hq + 2 * self.hk, self.d)
        q, k, v = qkv.split([self.hq, self.hk, self.hk], 1)
        q = hum.rotary_kv_write(self.kv, self.cache, q, k, v, pos, self.freq, slots, factor=self.factor, q_norm=self.w_q,
                                k_norm=self.w_k)
        return a, a_s, stream, qkv, q

    def rest(self, att, stream):
        o = hum.linear(self.do, self.po, att.flatten(1))
        y, stream = hum.rms_norm(o, self.w_post, residual=stream)
        logits = hum.linear(self.dr, self.pr, y)
        ids, w = hum.moe_route(logits, self.topk, bias=self.bias, **self.routing)
        return o, y, stream, logits, ids, w, hum.moe_gemm(self.d13, self.p13, self.d2, self.p2, y, ids, w)

    def step(self, x, stream, pos, slots, table, lens):
        a = self.append(x, stream, pos, slots)
        att = hum.kv_attention(self.kv, self.cache, a[4], table, lens)
        return a + (att,) + self.rest(att, a[2])

    def check_append(self, x, stream, pos, slots, out, before):
        """Against the oracle, from the cache's bytes before the call."""
        a, a_s, s1, qkv, q = out
        y, h = L.rms_norm(f64(x), f64(self.w_in), np.float32(1e-6), f64(stream))
        check_codes(a, a_s, y, "fp8_token")
        assert torch.equal(s1, (x.float() + stream.float()).to(torch.bfloat16))
        codes = oracle.formats.decode_e4m3(a.cpu().numpy()) * a_s.double().cpu().numpy()[:, None]
        assert_tol(qkv.flatten(1), oracle.gemm.linear(self.oq, codes, self.wqkv["codes"], self.wqkv["scales"]), "qkv")
        c = Append.__new__(Append)                       # its checks, on this cache
        c.fmt, c.t, c.hq, c.hk, c.d, c.r, c.ps, c.layout = self.fmt, len(pos), self.hq, self.hk, self.d, self.d, self.ps, "half"
        c.qkv, c.pos, c.slots, c.freq, c.pages = qkv, pos, slots, self.freq, self.kv.num_pages
        # slots that were written before hold what they held; the rest of the cache is 0xA5
        cache = self.cache.clone()
        keep = self.written[~torch.isin(self.written, slots)] if len(self.written) else self.written
        if len(keep):
            for x_before, x_after in zip(hum.kv_read(self.kv, before, keep), hum.kv_read(self.kv, self.cache, keep)):
                assert torch.equal(x_before, x_after)
            other = torch.full_like(cache, 0xA5)
            self._copy(cache, other, slots)
            cache = other
        c.check(q, cache, factor=float(np.float32(self.factor)), q_norm=self.w_q, k_norm=self.w_k)
        self.written = torch.cat([self.written, slots])

    def _copy(self, src, dst, slots):
        """The bytes of `slots` from one cache to another."""
        o = oracle.attention.Cache(self.fmt, self.kv.num_pages, self.ps, self.hk, self.d)
        s, t = (x.view(self.kv.num_pages, self.hk, -1) for x in (src, dst))
        for slot in slots.tolist():
            for which in (0, 1):
                code, sc = o._where(which, slot % self.ps)
                idx = torch.from_numpy(np.concatenate([np.arange(code, code + o.row), np.atleast_1d(sc).astype(np.int64)])).cuda()
                t[slot // self.ps][:, idx] = s[slot // self.ps][:, idx]

    def check_rest(self, att, s1, out):
        o, y, s2, logits, ids, w, moe = out
        assert_tol(o, oracle.gemm.linear(self.oo, f64(att.flatten(1)), self.wo["codes"], self.wo["scales"], self.wo["zeros"]), "o")
        _near(y, L.rms_norm(f64(o), f64(self.w_post), np.float32(1e-6), f64(s1))[0])
        assert torch.equal(s2, (o.float() + s1.float()).to(torch.bfloat16))
        assert_tol(logits, oracle.gemm.linear(self.our, f64(y), self.wr["codes"], self.wr["scales"]), "router")
        ri, rw = L.route(f64(logits), self.topk, bias=self.bias.double().cpu().numpy(), **self.routing)
        assert np.array_equal(ids.cpu().numpy(), ri)
        assert (np.abs(w.double().cpu().numpy() - rw) <= rw * (24 + 64) * 2.0 ** -24).all()
        ref = oracle.moe.moe_forward(self.o13, self.w13, self.o2, self.w2, bf16_bits_of(y), ids.cpu().numpy(), w.cpu().numpy(), "bf16")
        assert_tol(moe, ref, "experts")


def _x(seed, t, hid):
    return dev(synth.bf16_normal(synth.rng(seed), (t, hid)))


@pytest.mark.parametrize("fmt", ["bf16", "fp8_token", "mxfp8", "mxfp4"])
def test_prompt_and_decode_steps(fmt):
    ly = Layer(fmt, 40)
    ly.fmt, ly.written = fmt, torch.zeros(0, dtype=torch.int64, device="cuda")
    lens = np.array([37, 1, 90])
    table = np.random.default_rng(1).permutation(40)[:30].reshape(3, 10).astype(np.int32)
    slots_of = lambda seq, pos: table[seq, pos // ly.ps].astype(np.int64) * ly.ps + pos % ly.ps  # noqa: E731
    seq, pos = np.repeat(np.arange(3), lens), np.concatenate([np.arange(n) for n in lens])
    x, stream = _x(1, len(pos), ly.hid), _x(2, len(pos), ly.hid)
    before = ly.cache.clone()
    out = ly.append(x, stream, dev(pos), dev(slots_of(seq, pos)))
    ly.check_append(x, stream, dev(pos), dev(slots_of(seq, pos)), out, before)
    att = out[4].contiguous()                            # (a prompt's own attention is not this library's: any rows do)
    ly.check_rest(att, out[2], ly.rest(att, out[2]))
    for s in range(3):
        pos, lens = lens.copy(), lens + 1
        slots = dev(slots_of(np.arange(3), pos))
        x, stream, before = _x(10 + s, 3, ly.hid), _x(20 + s, 3, ly.hid), ly.cache.clone()
        out = ly.step(x, stream, dev(pos), slots, dev(table), dev(lens.astype(np.int32)))
        ly.check_append(x, stream, dev(pos), slots, out[:5], before)
        c = Attention.__new__(Attention)
        ref = oracle.attention.Cache(fmt, 40, ly.ps, ly.hk, ly.d)
        ref.buf = ly.cache.cpu().numpy().reshape(ref.buf.shape)
        c.cache, c.table, c.d, c.q, c.lens = ref, table, ly.d, f64(out[4]), lens
        got = hum.kv_attention(ly.kv, ly.cache, out[4], dev(table), dev(lens.astype(np.int32)), return_lse=True)
        assert torch.equal(got[0], out[5])
        c.check(got, what=f"step {s}")
        ly.check_rest(out[5], out[2], out[6:])


@pytest.mark.parametrize("fmt", ["fp8_token", "mxfp4"])
def test_captured_step_replays_with_growing_sequences(fmt):
    """One captured step replayed while its inputs change in place, against eager steps on a second cache."""
    ly, eager = Layer(fmt, 40), Layer(fmt, 40)
    table = torch.arange(30, dtype=torch.int32, device="cuda").view(2, 15)
    x, stream = (torch.zeros((2, ly.hid), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pos = torch.zeros(2, dtype=torch.int64, device="cuda")
    slots, lens = torch.zeros_like(pos), torch.zeros(2, dtype=torch.int32, device="cuda")

    def feed(s, n0):
        x.copy_(_x(300 + s, 2, ly.hid))
        stream.copy_(_x(400 + s, 2, ly.hid))
        pos.copy_(torch.tensor(n0))
        slots.copy_(table.gather(1, (pos // ly.ps)[:, None]).squeeze(1).long() * ly.ps + pos % ly.ps)
        lens.copy_(pos + 1)

    feed(0, [0, 0])
    for _ in range(2):
        ly.step(x, stream, pos, slots, table, lens)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = ly.step(x, stream, pos, slots, table, lens)
    for s in range(30):
        feed(s, [s, s * 5])
        want = eager.step(x, stream, pos, slots, table, lens)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(res, want):
            assert torch.equal(a, b), s
    assert torch.equal(ly.cache, eager.cache)


def test_calls_on_two_streams_at_once():
    """Nothing is shared between calls: they give on side streams, overlapping, what they gave alone."""
    ly = [Layer(f, 60) for f in ("bf16", "mxfp8")]
    t = 700
    args = [(_x(50 + i, t, 256), _x(60 + i, t, 256), torch.arange(t, device="cuda"), torch.arange(t, device="cuda") + 16 * i)
            for i in range(2)]
    logits = [torch.randn(3000, 256, generator=torch.Generator("cuda").manual_seed(i), device="cuda") for i in range(2)]
    want = [(y.append(*a), hum.moe_route(lg, 8, "sigmoid", num_groups=8, topk_groups=4, group_score="top2"))
            for y, a, lg in zip(ly, args, logits)]
    caches = [y.cache.clone() for y in ly]
    for y in ly:
        y.cache.fill_(0xA5)
    streams = [torch.cuda.Stream() for _ in ly]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for y, a, lg, s in zip(ly, args, logits, streams):
            with torch.cuda.stream(s):
                got.append((y.append(*a), hum.moe_route(lg, 8, "sigmoid", num_groups=8, topk_groups=4, group_score="top2")))
    torch.cuda.synchronize()
    for g, w, y, c in zip(got, want, ly, caches):
        assert all(torch.equal(a, b) for a, b in zip(g[0] + g[1], w[0] + w[1])) and torch.equal(y.cache, c)


def test_padding_tokens_route_nowhere():
    """Rows of -inf logits: no expert, and nothing from the expert layer, whatever the rows hold."""
    ly = Layer("bf16", 8)
    y = _x(5, 9, ly.hid)
    logits = hum.linear(ly.dr, ly.pr, y)
    logits[[2, 8]] = -float("inf")
    y[2] = float("nan")
    ids, w = hum.moe_route(logits, ly.topk, bias=ly.bias, **ly.routing)
    out = hum.moe_gemm(ly.d13, ly.p13, ly.d2, ly.p2, y, ids, w)
    assert (ids[[2, 8]] == -1).all() and (out[[2, 8]] == 0).all()
    keep = [0, 1, 3, 4, 5, 6, 7]
    ref = oracle.moe.moe_forward(ly.o13, ly.w13, ly.o2, ly.w2, bf16_bits_of(y[keep]), ids[keep].cpu().numpy(), w[keep].cpu().numpy(), "bf16")
    assert_tol(out[keep], ref, "experts")


def test_norm_feeds_every_stage_in_place():
    """The residual stream kept in one buffer over a layer, in place, equals the calls out of place."""
    ly = Layer("bf16", 8)
    x, stream = _x(6, 5, ly.hid), _x(7, 5, ly.hid)
    buf = stream.clone()
    y1, s1 = hum.rms_norm(x, ly.w_in, residual=stream)
    y2, s2 = hum.rms_norm(x.clone(), ly.w_in, residual=buf, residual_out=buf)
    assert s2 is buf and torch.equal(y1, y2) and torch.equal(s1, buf)
    assert np.abs(f64(y1)).max() > EPS
