"""The linear layer's direct global->LDS loads, formed on the CPU the way the kernel forms
them (thread -> row, chunk, swizzled place, stage): every place of a half tile receives the
element that its reader expects, or a zero from an offset past the buffer's end; no
offset wraps; and the readers of a fragment meet no bank twice."""
import numpy as np
import pytest

OOB = 0x80000000


def _f(w, k):
    return (k & 3) | (((k >> 3) & 1) << 2) if w >= 128 else ((k >> 1) & 1) | (((k >> 3) & 1) << 1)


def _place(w, kmaj, row, c):
    return c ^ ((row >> 1) & 7) if kmaj else c ^ (2 * _f(w, row))


def _half(w, kmaj, r0, rows, ld, h, kt, K, nbytes):
    """What each 16-byte place of half h of stage kt holds: the flat element index of its first
    element, or -1 for zeros."""
    per, cpr = w * 128 // 8192, (128 if kmaj else 2 * w) // 16
    rstep, ld2 = 512 // cpr, 2 * ld
    out = np.full(w * 8, -2, dtype=np.int64)
    for tid in range(512):
        row = tid // cpr
        c = _place(w, kmaj, row, tid % cpr)
        base = ((r0 + row) * ld + 8 * c) * 2 if kmaj else (row * ld + r0 + 8 * c) * 2
        kk = 8 * c if kmaj else (row if r0 + h * w + 8 * c < rows else 2 ** 31 - 1)
        at = kt * 128 + h * w * ld2 if kmaj else kt * 64 * ld2 + h * 2 * w
        for i in range(per):
            ok = kk < K - kt * 64 - (0 if kmaj else i * rstep)
            off = base + at + i * rstep * ld2 if ok else OOB
            assert off < 2 ** 32 and off % 16 == 0
            place = i * 512 + tid
            assert out[place] == -2
            out[place] = off // 2 if off + 16 <= nbytes else -1
            assert off >= nbytes or off + 16 <= nbytes
    return out


@pytest.mark.parametrize("w", [64, 128])
@pytest.mark.parametrize("rows,K", [(8, 8), (200, 72), (264, 136), (520, 64), (128, 200)])
def test_k_major_places(w, rows, K):
    for r0 in range(0, rows, 2 * w):
        for kt in range((K + 63) // 64 + 2):
            for h in range(2):
                got = _half(w, True, r0, rows, K, h, kt, K, rows * K * 2)
                for r in range(w):
                    for c in range(8):
                        row, k = r0 + h * w + r, kt * 64 + 8 * c
                        want = row * K + k if row < rows and k < K else -1
                        assert got[r * 8 + _place(w, True, r, c)] == want


@pytest.mark.parametrize("w", [64, 128])
@pytest.mark.parametrize("cols,K", [(8, 1), (200, 77), (264, 130), (520, 64), (128, 201)])
def test_mn_major_places(w, cols, K):
    for c0 in range(0, cols, 2 * w):
        for kt in range((K + 63) // 64 + 2):
            for h in range(2):
                got = _half(w, False, c0, cols, cols, h, kt, K, K * cols * 2)
                for r in range(64):
                    for c in range(w // 8):
                        col, k = c0 + h * w + 8 * c, kt * 64 + r
                        want = k * cols + col if col < cols and k < K else -1
                        assert got[r * (w // 8) + _place(w, False, r, c)] == want


@pytest.mark.parametrize("w", [64, 128])
def test_fragment_reads_meet_no_bank_twice(w):
    """16 lanes of a 16-byte read, and 32 lanes of a transposing 8-byte read, cover 256 bytes of
    banks once each."""
    for r0 in range(0, w, 16):
        for step in range(2):
            for g in range(4):
                banks = [(((r0 + j) * 128 + (_place(w, True, r0 + j, 4 * step + g) << 4)) // 16) % 16 for j in range(16)]
                assert len(set(banks)) == 16
            for half in range(2):
                seen = []
                for lane in range(32 * half, 32 * half + 32):
                    j = lane & 15
                    k, col = 32 * step + 8 * (lane >> 4) + (j >> 2), r0 + 4 * (j & 3)
                    seen.append(((k * 2 * w + (_place(w, False, k, col >> 3) << 4) + (col & 7) * 2) // 8) % 32)
                assert len(set(seen)) == 32
