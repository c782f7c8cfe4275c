"""mc_grouped_tile: the tile that a product's sizes choose, and its refusals (no GPU)."""
import ctypes as C

from expert_cache_offloaded_amd import _lib as L


def tile(**kw):
    keep = (C.c_uint8 * 4112)()
    p = (C.addressof(keep) + 15) & ~15
    d = dict(x_fmt=0, w_fmt=1, y_fmt=0, swiglu=0, E=1, M=2, N=64, K=64, x_rows=2, x_div=1, y_rows=2, ldx=64, ldy=64, n=1,
             x=p, x_scale=p, w=p, w_scale=p, y=p, y_scale=p, offsets=p)
    d.update(kw)
    out = (C.c_int32 * 3)(-1, -1, -1)
    rc = L.lib().mc_grouped_tile(C.byref(L.Grouped(**d)), out)
    return tuple(out) if rc == L.MC_OK else rc


def test_tiles_by_size():
    def dense(M, N, K):
        return tile(offsets=None, M=M, N=N, K=K, ldx=K, ldy=N, x_rows=M, y_rows=M)
    assert tile() == (16, 0, 1)
    assert dense(16, 4096, 4096) == (16, 0, 1)
    assert dense(17, 4096, 2048) == (64, 64, 4)
    assert dense(333, 4100, 2080) == (64, 64, 2)
    assert dense(1000, 4096, 2080) == (128, 128, 2)
    assert dense(8192, 4096, 4096) == (256, 256, 1)
    # one matrix of more than 4 GiB
    assert dense(300, 1 << 17, 1 << 17) == (16, 0, 1)


def test_refusals():
    assert tile(K=48) == L.MC_EINVAL and "mc_grouped_tile" in L.last_error()
    assert L.lib().mc_grouped_tile(None, (C.c_int32 * 3)()) == L.MC_EINVAL
    assert L.lib().mc_grouped_tile(C.byref(L.Grouped()), None) == L.MC_EINVAL
