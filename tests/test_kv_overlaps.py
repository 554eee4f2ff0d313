"""Outputs of the attention and of the cache's read that lie in what the call
reads: refused before any launch.  The CPU test's addresses are never touched:
every call there ends in a refusal."""
import ctypes

import pytest
import torch

import quantized_gemm_packed_amd as hum

P = ctypes.c_void_p


def test_attention_outputs_inside_inputs_are_refused():
    lib = hum.load_library()
    d = hum.make_kv_desc("fp8_token", 6, 16, 2, 64)
    nb, need = hum.kv_cache_bytes(d), hum.kv_attention_workspace_bytes(d, 4, 3, 2)
    q, cache, out, ws, tab, lens, lse = (1 << 20) + 768, 2 << 20, 3 << 20, 4 << 20, 12 << 20, 13 << 20, 14 << 20

    def call(c=cache, q=q, qts=512, tab=tab, lens=lens, out=out, lse=lse, ws=ws):
        return lib.hum_kv_attention(ctypes.addressof(d), P(c), nb, 4, 3, P(q), qts, 64, P(tab), 2, 2, P(lens), 0, 1.0, P(out),
                                    P(lse), P(ws), need, None)
    for kw in (dict(out=q), dict(out=q + 512 * 2), dict(out=q - 1536 + 16), dict(q=out, qts=512), dict(q=out + 2, qts=256),
               dict(out=cache + nb - 16), dict(out=cache - 1536 + 16), dict(tab=out + 1532), dict(lens=out + 8),
               dict(lse=out + 1532), dict(lse=out - 44), dict(lse=cache), dict(lse=tab + 20), dict(lse=lens + 8),
               dict(lse=q + 2 * 1024 + 508), dict(out=ws + need - 16), dict(lse=ws), dict(ws=out + 1520), dict(ws=cache + nb - 16),
               dict(lens=ws), dict(tab=ws + need - 4), dict(ws=q - q % 16)):
        assert call(**kw) == 1, kw
        assert b"overlap" in lib.hum_last_error()


def test_read_outputs_inside_the_cache_or_the_slots_are_refused():
    lib = hum.load_library()
    d = hum.make_kv_desc("bf16", 6, 16, 2, 64)
    a, nb = ctypes.addressof(d), hum.kv_cache_bytes(d)
    cache, slots, k, v = 1 << 20, 2 << 20, 3 << 20, 4 << 20
    for s, x, y in ((slots, cache, v), (slots, k, cache + nb - 16), (slots, cache - 752, v), (k + 760, k, v), (v, k, v)):
        assert lib.hum_kv_read(a, P(cache), nb, 3, P(s), P(x), P(y), None) == 1, (s, x, y)
        assert b"overlap" in lib.hum_last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("lens,hq,hk,d", [([300, 1, 0, 5000], 8, 2, 128), ([20011], 4, 1, 64), ([70] * 90, 40, 1, 64)])
def test_attention_into_its_own_queries(lens, hq, hk, d):
    """out may be q itself: a row's last reader is past it when it is stored, also where a head is cut into parts."""
    from test_gpu_kv import Case
    c = Case(31, "bf16", lens, hq, hk, d, 16)
    want = c.run(return_lse=True)
    for _ in range(3):
        q = c.dev["q"].clone()
        out, lse = c.run(q=q, out=q, return_lse=True)
        assert out is q and torch.equal(q, want[0]) and torch.equal(lse, want[1])


@pytest.mark.gpu
def test_binding_refuses_shifted_outputs():
    from test_gpu_kv import Case
    c = Case(32, "bf16", [40, 7], 4, 2, 64, 16)
    flat = torch.randn(2 * 4 * 64 + 256, device="cuda").to(torch.bfloat16)
    before, cache = flat.clone(), c.dev["cache"].clone()
    with pytest.raises(hum.HumError, match="overlap"):
        c.run(q=flat[:512].view(2, 4, 64), out=flat[256:768].view(2, 4, 64))
    inside = c.dev["cache"][:2 * 4 * 64 * 2].view(torch.bfloat16).view(2, 4, 64)
    with pytest.raises(hum.HumError, match="overlap"):
        c.run(out=inside)
    with pytest.raises(hum.HumError, match="overlap"):
        hum.kv_read(c.desc, c.dev["cache"], torch.arange(2, device="cuda"), k_out=inside[:, :2].contiguous().clone(),
                    v_out=c.dev["cache"][1024:1024 + 512].view(torch.bfloat16).view(2, 2, 64))
    torch.cuda.synchronize()
    assert torch.equal(flat, before) and torch.equal(c.dev["cache"], cache)


@pytest.mark.gpu
def test_rows_of_the_cache_are_moved_to_other_slots():
    """k and v of a write may be views of the (bf16) cache: one page's tokens into another's slots."""
    pages, ps, hk, d = 4, 32, 3, 128
    desc = hum.make_kv_desc("bf16", pages, ps, hk, d)
    cache = torch.randn(hum.kv_cache_bytes(desc) // 2, device="cuda").to(torch.bfloat16)
    rows = cache.view(pages, hk, 2, ps, d)
    want = rows.clone()
    want[3] = want[1]
    k, v = (rows[1, :, i].transpose(0, 1) for i in (0, 1))
    hum.kv_write(desc, cache.view(torch.uint8), k, v, torch.arange(3 * ps, 4 * ps, device="cuda"))
    assert torch.equal(rows, want)
