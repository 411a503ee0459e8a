"""Which memory the 8-bit path's and the norm's calls take in two roles: told from
the addresses on the host, before any of them is looked at."""

import ctypes
import random

import pytest

BASE = 1 << 40


@pytest.fixture(scope="module")
def lib(built_library):
    from lm_head_exact_gb300 import binding
    return binding.library()


def P(at):
    return ctypes.c_void_p(at)


def _refused(lib, status):
    """Whether a call that fails in any case (these addresses are nobody's)
    fails for what overlaps."""
    assert status != 0
    return "overlaps" in lib.fs_last_error().decode()


def _bytes(at, rows, width, pitch):
    return {at + r * pitch + i for r in range(rows) for i in range(width)}


def test_matrices_that_share_a_byte(lib):
    """Against sets of addresses: rows of one pitch may lie side by side, whatever
    their number and order; without a common pitch, one may lie behind the other."""
    rng = random.Random(5)
    seen = [0, 0]
    for _ in range(4000):
        rows, cols = rng.choice((1, 2, 3, 5)), rng.choice((1, 3, 8))
        pitch = 16 * rng.choice((1, 2, 3))
        x_stride = pitch // 2 if rng.random() < 0.7 else cols + rng.randrange(5)
        x = BASE + 2 * rng.randrange(-60, 100)
        call = lambda q, s: lib.fs_quantize_fp8(P(x), 1, rows, cols, x_stride, 0, 1, 3, P(q), pitch, P(s), 1, rows, P(0))  # noqa: E731
        xs, q = _bytes(x, rows, 2 * cols, 2 * x_stride), BASE + 16 * rng.randrange(5)
        qs = _bytes(q, rows, cols, pitch)
        got = _refused(lib, call(q, BASE + (1 << 20)))
        if rows == 1 or 2 * x_stride == pitch or max(xs) < min(qs) or max(qs) < min(xs):
            assert got == bool(xs & qs), (rows, cols, pitch, x_stride, x - q)
            seen[got] += 1
        else:
            assert got                                         # between each other's ends
    assert min(seen) > 300


def test_scales_beside_their_rows(lib):
    """A row's scales right behind its bytes are no one else's; on them they are."""
    def call(s_at, s_row, s_col, rows=6, cols=300):
        return _refused(lib, lib.fs_quantize_fp8(P(BASE), 1, rows, cols, cols, 0, 1, 3, P(BASE + 65536), 336, P(BASE + 65536 + s_at),
                                                 s_row, s_col, P(0)))
    assert not call(304, 84, 1) and not call(6 * 336, 3, 1) and not call(6 * 336, 1, 6)
    assert call(296, 84, 1) and call(328, 84, 1) and call(0, 1, 6) and call(5 * 336, 3, 1)
    assert call(-65536, 3, 1)                                  # on x


def test_product(lib):
    m, n, k = 5, 7, 300
    a, b, asc, bsc, out = BASE, BASE + 65536, BASE + 131072, BASE + 196608, BASE + 262144

    def call(out=out, out_stride=n, b_block=1):
        return _refused(lib, lib.fs_fp8_matmul(P(a), 3, 304, P(asc), 1, m, P(b), 3, 304, P(bsc), 3, 1, b_block, m, n, k, P(out), 0,
                                               out_stride, P(0)))
    assert not call()
    for at, rows, block in ((a, m, 1), (b, n, 1), (asc, 1, 1), (bsc, 1, 1), (bsc, 1, 128)):
        assert call(at, b_block=block) and call(at - 4 * (m * n - 1), b_block=block) and not call(at - 4 * m * n, b_block=block)
    assert call(bsc + 4 * 3 * n - 4) and not call(bsc + 4 * 3 * n)
    assert call(bsc + 8, b_block=128) and not call(bsc + 12, b_block=128)


def _norm(lib, x=BASE, y=BASE + (1 << 20), q=0, scale=0, weight=BASE + (2 << 20), bias=BASE + (3 << 20), mean=BASE + (4 << 20),
          rstd=BASE + (5 << 20), n=6, d=40, x_stride=48, y_stride=48, rms=0):
    return _refused(lib, lib.fs_layer_norm(P(x), 1, n, d, x_stride, P(weight), P(bias), 0, rms, 1e-5, P(y), y_stride, P(mean),
                                           P(rstd), P(q), 3, 48, P(scale), 1, n, P(0)))


def test_norm(lib):
    x, y, weight, bias, mean, rstd = (BASE + (i << 20) for i in range(6))
    assert not _norm(lib) and not _norm(lib, y=x)
    assert not _norm(lib, x=x + 80, y=x, x_stride=96, y_stride=96)       # two halves of one matrix
    assert _norm(lib, y=x + 96) and _norm(lib, y=x + 2) and _norm(lib, y=x, y_stride=64)
    assert not _norm(lib, y=x, y_stride=64, n=1)                         # one row has no pitch
    for at, size in ((weight, 160), (bias, 160)):
        assert _norm(lib, y=at) and _norm(lib, y=at + size - 2) and not _norm(lib, y=at + size)
        assert _norm(lib, mean=at) and _norm(lib, rstd=at + size - 4)
        assert _norm(lib, y=0, q=at, scale=rstd + 65536) and _norm(lib, y=0, q=y, scale=at)
    for at in (x, y, rstd):
        assert _norm(lib, mean=at)
        assert not _norm(lib, mean=at, rms=1)                            # not written then
    assert _norm(lib, rstd=x + 4) and _norm(lib, rstd=y + 4 * 96 + 40)
    assert _norm(lib, y=0, q=x, scale=y) and _norm(lib, y=0, q=y, scale=y) and _norm(lib, y=0, q=y, scale=x)
    assert _norm(lib, y=0, q=y, scale=rstd) and _norm(lib, y=0, q=rstd, scale=y)
    assert not _norm(lib, y=0, q=y, scale=rstd + 24)


def _back(lib, g=BASE, x=BASE + (1 << 20), weight=BASE + (2 << 20), mean=BASE + (3 << 20), rstd=BASE + (4 << 20),
          gx=BASE + (5 << 20), gw=BASE + (6 << 20), gb=BASE + (7 << 20), work=0, size=0, n=6, d=40, gx_stride=48, rms=0):
    return _refused(lib, lib.fs_layer_norm_backward(P(g), 48, P(x), 1, n, d, 48, P(weight), 0, rms, P(mean), P(rstd), P(gx),
                                                    gx_stride, P(gw), P(gb), P(work), size, P(0)))


def test_norm_gradients(lib):
    g, x, weight, mean, rstd, gx, gw, gb, work = (BASE + (i << 20) for i in range(9))
    assert not _back(lib) and not _back(lib, gx=g) and not _back(lib, gx=x)
    assert not _back(lib, g=x, gx=x) and _back(lib, g=x + 96, gx=x)
    assert _back(lib, gx=g + 96) and _back(lib, gx=x - 96) and _back(lib, gx=x, gx_stride=64)
    for at in (mean, rstd, weight):
        assert _back(lib, gx=at) and _back(lib, gw=at) and _back(lib, gb=at - 8)
    assert not _back(lib, gx=mean, rms=1)                                # not read then
    for at in (g, x, gx):
        assert _back(lib, gw=at + 96) and _back(lib, gb=at + 96)
    assert _back(lib, gb=gw + 156) and not _back(lib, gb=gw + 160) and _back(lib, gb=gw)
    need = lib.fs_layer_norm_backward_workspace_bytes(6, 40)
    assert not _back(lib, work=work, size=need)
    for at in (g, x, weight, mean, rstd, gx, gw, gb):
        assert _back(lib, work=at, size=need) and _back(lib, work=at - need + 4, size=need)
        assert not _back(lib, work=at - need, size=need)
        assert not _back(lib, work=at, size=need, gw=0, gb=0)            # no sums, no workspace


def test_sizes_beyond_64_bits(lib):
    """Rows times a stride may pass 2^64 before they are found not to be memory."""
    big = (1 << 40) - 16
    assert _refused(lib, lib.fs_quantize_fp8(P(BASE + 32), 1, (1 << 31) - 1, 8, 8, 0, 1, 3, P(BASE), big, P(BASE + 64), 1, 1 << 31, P(0)))
