"""4-bit pools, weight gathering and eviction without a GPU: descriptors,
workspace sizes, and every refusal before the first CUDA call."""
import ctypes

import pytest

import paged_kv_cache_478_b200 as pa

OK = ctypes.c_void_p(0x2000)  # aligned, never dereferenced on these paths
ODD = ctypes.c_void_p(0x2008)
F = ctypes.c_float


@pytest.mark.parametrize("code", [pa.PA_Q4_F16, pa.PA_Q4_BF16])
@pytest.mark.parametrize("dim", [64, 128])
def test_descriptor(code, dim):
    p = pa.pa_pool_create(100, 16, 3, dim, code)
    assert (p.dtype, p.elem_bytes, p.head_stride, p.block_stride) == (code, 2, 9 * dim, 27 * dim)
    assert p.bytes_per_pool == 100 * 27 * dim
    pa.pa_pool_set_query_heads(p, 24)
    assert p.q_per_kv == 8
    assert pa.pa_decode_workspace_bytes(p, 4, 8) > 0


@pytest.mark.parametrize("args,status", [
    ((100, 16, 3, 96, pa.PA_Q4_F16), 2), ((100, 8, 3, 64, pa.PA_Q4_BF16), 2),
    ((100, 16, 3, 64, 5), 2), ((0, 16, 3, 64, pa.PA_Q4_F16), 1)])
def test_descriptor_refusals(args, status):
    with pytest.raises(pa.PagedAttnError) as e:
        pa.pa_pool_create(*args)
    assert e.value.status == status


def test_paths_without_a_4_bit_form_refuse():
    lib, p = pa.lib(), pa.pa_pool_create(16, 16, 2, 64, pa.PA_Q4_F16)
    st = lib.pa_prefill_attention(ctypes.byref(p), OK, OK, OK, OK, 4, OK, OK, 1, 8, 8, 0, F(0.1), OK, None)
    assert st == 2 and b"pa_convert_blocks" in lib.pa_last_error()
    st = lib.pa_decode_attention_shared_prefix(ctypes.byref(p), OK, OK, OK, OK, 4, OK, 1, OK, OK, 1,
                                               OK, 1, 1, 1, 0, F(0.1), OK, OK, 1 << 20, 0, None)
    assert st == 2


def test_convert_blocks_refusals():
    lib = pa.lib()
    mk = lambda *a: pa.pa_pool_create(*a)  # noqa: E731
    f16, q16 = mk(8, 16, 2, 64, pa.PA_F16), mk(8, 16, 2, 64, pa.PA_Q4_F16)
    bf, f32, qbf = (mk(8, 16, 2, 64, c) for c in (pa.PA_BF16, pa.PA_F32, pa.PA_Q4_BF16))
    other = mk(8, 16, 3, 64, pa.PA_Q4_F16)

    def call(a, b, ks=OK, vd=OK, pairs=OK, n=1):
        return lib.pa_convert_blocks(ctypes.byref(a), ks, OK, ctypes.byref(b), OK, vd, pairs, n, None)

    for a, b in [(f16, f16), (q16, q16), (bf, q16), (f32, q16), (qbf, f16), (q16, f32)]:
        assert call(a, b) == 2, (a.dtype, b.dtype)
    assert call(f16, other) == 1 and call(f16, q16, n=-1) == 1
    assert call(f16, q16, ks=None) == 1 and call(f16, q16, pairs=None) == 1 and call(f16, q16, vd=ODD) == 1
    assert call(f16, q16, n=0) == 0
    assert lib.pa_convert_blocks(None, OK, OK, ctypes.byref(q16), OK, OK, OK, 1, None) == 1


def test_append_and_copy_refusals():
    lib, p = pa.lib(), pa.pa_pool_create(16, 16, 2, 64, pa.PA_Q4_F16)
    assert lib.pa_reshape_and_cache(ctypes.byref(p), OK, ODD, OK, 1, OK, OK, None) == 1
    assert lib.pa_reshape_and_cache(ctypes.byref(p), OK, OK, None, 1, OK, OK, None) == 1
    assert lib.pa_reshape_and_cache(ctypes.byref(p), OK, OK, OK, 0, OK, OK, None) == 0
    assert lib.pa_copy_blocks(ctypes.byref(p), OK, ODD, OK, 1, None) == 1


def test_mass_workspace_covers_the_scores():
    p = pa.pa_pool_create(4096, 16, 4, 128, pa.PA_F16)
    pa.pa_pool_set_query_heads(p, 8)
    base, mass = pa.pa_decode_workspace_bytes(p, 3, 7, 100), pa.pa_decode_mass_workspace_bytes(p, 3, 7, 100)
    assert mass >= base + 3 * 8 * 100 * 4 + 3 * 8 * 4
    with pytest.raises(pa.PagedAttnError):
        pa.pa_decode_mass_workspace_bytes(p, 3, 7, 100, 24)


def test_mass_refusals():
    lib, p = pa.lib(), pa.pa_pool_create(16, 16, 2, 64, pa.PA_F32)

    def call(q=OK, lens=OK, S=1, scale=0.1, mass_out=OK, stride=64, decay=1.0, blocks=4):
        return lib.pa_decode_attention_mass(ctypes.byref(p), q, OK, OK, OK, blocks, lens, S, 0, F(scale), OK,
                                            None, mass_out, stride, F(decay), OK, 1 << 20, 0, None)

    assert call(q=None) == 1 and call(lens=None) == 1 and call(S=-1) == 1 and call(blocks=0) == 1
    assert call(mass_out=None) == 1 and call(stride=63) == 1 and call(S=65536) == 1
    assert call(decay=float("nan")) == 1 and call(scale=float("inf")) == 1
    assert call(S=0) == 0
    st = lib.pa_decode_attention_mass_planned(ctypes.byref(p), OK, OK, OK, OK, 4, 1, 0, F(0.1), OK, None, None,
                                              64, F(1), OK, 1 << 20, 0, None)
    assert st == 1


def test_evict_refusals():
    lib, p = pa.lib(), pa.pa_pool_create(16, 16, 2, 64, pa.PA_F16)
    good = pa.pa_track(0x2000, 0x3000, 0x4000, 64)

    def call(track=good, out=good, S=1, k=OK, keep=OK, sinks=0, recent=0, ws=OK, size=1 << 20, blocks=4):
        return lib.pa_evict_tokens(ctypes.byref(p), k, OK, OK, blocks, OK, S, keep, sinks, recent,
                                   ctypes.byref(track), ctypes.byref(out), 0, ws, size, None)

    assert call(k=None) == 1 and call(k=ODD) == 1 and call(keep=None) == 1 and call(S=-1) == 1
    assert call(sinks=-1) == 1 and call(recent=-1) == 1 and call(blocks=0) == 1 and call(S=65536) == 1
    assert call(track=pa.pa_track(0x2000, 0x3000, 0x4000, 63)) == 1
    assert call(out=pa.pa_track(0x2000, 0x9000, 0x4000, 65)) == 1  # in place, another stride
    assert call(out=pa.pa_track(None, 0x3000, 0x4000, 64)) == 1
    assert call(ws=None) == 6 and call(ws=ODD) == 6
    need = pa.pa_evict_workspace_bytes(p, 1, 4)
    assert call(size=need - 1) == 6
    assert call(S=0) == 0


def test_sizes_beyond_the_kernels_indexes_are_refused():
    lib, p = pa.lib(), pa.pa_pool_create(16, 16, 2, 64, pa.PA_Q4_F16)
    n = ctypes.c_size_t()
    ask = lambda pool, S, blocks: lib.pa_evict_workspace_bytes(ctypes.byref(pool), S, blocks, 0, ctypes.byref(n))  # noqa: E731
    assert ask(p, 65535, 1 << 26) == 0 and n.value >= 65535 * (1 << 29) * 8
    assert ask(p, 65536, 4) == 1 and ask(p, 1, (1 << 26) + 1) == 2
    assert lib.pa_decode_mass_workspace_bytes(ctypes.byref(p), 65536, 4, 0, 0, ctypes.byref(n)) == 1
    t = pa.pa_track(0x2000, 0x3000, 0x4000, 1 << 31)
    assert lib.pa_evict_tokens(ctypes.byref(p), OK, OK, OK, (1 << 26) + 1, OK, 1, OK, 0, 0, ctypes.byref(t), ctypes.byref(t),
                               0, OK, 1 << 40, None) == 2
    with pytest.raises(pa.PagedAttnError):  # slots are 32-bit numbers
        pa.pa_pool_create(1 << 27, 16, 1, 64, pa.PA_Q4_F16)


def test_tensors_of_another_device_are_refused(monkeypatch):
    """The launch goes to the current device: a tensor elsewhere is refused before any call."""
    import torch

    class Elsewhere(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return 1

    t = torch.zeros(4).as_subclass(Elsewhere)
    pa._torch()
    monkeypatch.setattr(pa, "_current_device", lambda: 0)
    with pytest.raises(ValueError, match="current CUDA device"):
        pa._dev_ptr(t, "t")
    monkeypatch.setattr(pa, "_current_device", lambda: 1)
    assert pa._dev_ptr(t, "t") == t.data_ptr()
