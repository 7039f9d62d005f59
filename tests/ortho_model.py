"""The orthogonalised update by its definition in 64 bits, and with the kernel's roundings put in, each of which a
test can make coarser to see whether it would notice."""
from __future__ import annotations

import ctypes
import math
import os
import subprocess

import torch

ABC = (3.4445, -4.7750, 2.0315)


def _turned(G):
    X = G.double()
    return (X.t().contiguous(), True) if X.shape[0] > X.shape[1] else (X, False)


def defined(G, steps=5, abc=ABC, eps=1e-7, dtype=torch.float64):
    """With ``dtype`` float32: the plain form in 32 bits."""
    a, b, c = abc
    X, tall = _turned(G)
    X = (X / (X.norm() + eps)).to(dtype)
    for _ in range(steps):
        A = X @ X.t()
        X = a * X + (b * A + c * A @ A) @ X
    return (X.t() if tall else X).double()


def peak(abc, m):
    """The largest |a s + b s^3 + c s^5| of s from 0 to m."""
    a, b, c = abc
    s = torch.linspace(0, m, 200001, dtype=torch.float64)
    return float((s * (a + s * s * (b + c * s * s))).abs().max())


def scales(steps, abc):
    """Powers of two that fp16 holds X, the off-diagonal part of A and that of B times, at most 2^14, 2^10 and 2^8
    and such that what the coefficients can make of singular values up to 1 stays below 2^15."""
    a, b, c = abc
    m, x, o, p = 1.0, 0.0, 0.0, 0.0
    for _ in range(steps):
        x, o = max(x, m), max(o, m * m)
        t = torch.linspace(0, m * m, 200001, dtype=torch.float64)
        p = max(p, float((t * (b + c * t)).abs().max()))
        m = peak(abc, m) * (1 + 2.0 ** -8)

    def power(v, most):
        return 2.0 ** (most if v == 0 else min(most, math.floor(15 - math.log2(v))))

    return power(x, 14), power(o, 10), power(p, 8)


def values(steps, abc):
    """The largest |X|, |A| and |B| before each step, of singular values from 0 to 1 in exact arithmetic."""
    a, b, c = abc
    s = torch.linspace(0, 1, 100001, dtype=torch.float64)
    for _ in range(steps):
        t = s * s
        yield float(s.abs().max()), float(t.max()), float((t * (b + c * t)).abs().max())
        s = s * (a + t * (b + c * t))


def takes_rest(r, steps, abc):
    """Whether B X takes what fp16 leaves of X too."""
    return r <= 64 or abs(abc[0]) ** steps > r


MUTATIONS = ("diagonal of A in fp16", "diagonal of B in fp16", "no rest of X", "rest of X in 8 bits", "B X without the rest")


def rounded(G, steps=5, abc=ABC, eps=1e-7, mutation=None):
    """With the kernel's roundings: X as fp16 and what that leaves in fp16, the diagonals of A and B in fp32, the
    rest of them in fp16, sums in fp32.  ``mutation``: one of MUTATIONS."""
    a, b, c = abc
    X, tall = _turned(G)
    S, so, sb = scales(steps, abc)
    rest = takes_rest(min(G.shape), steps, abc) and mutation != "B X without the rest"
    V = (X * (S / (float(X.norm()) + eps))).float()   # X times S

    def half(v, s):
        return (v * s).half().float() / s

    for _ in range(steps):
        hi = V.half().float()
        lo = (V - hi).half().float()
        if mutation == "no rest of X":
            lo = torch.zeros_like(lo)
        elif mutation == "rest of X in 8 bits":   # times what keeps it in e4m3's range up to |X| = 1.3
            up = 2.0 ** 19 / S
            lo = ((V - hi) * up).clamp(-448, 448).to(torch.float8_e4m3fn).float() / up
        A = (hi @ hi.t()) * (1 / S ** 2)
        D = A.diagonal().clone()
        if mutation == "diagonal of A in fp16":
            D = half(D, so)
        O = half(A - torch.diag(A.diagonal()), so)
        OO = O @ O
        B = b * O + c * (OO + (D[:, None] + D[None, :]) * O)
        E = a + b * D + c * (OO.diagonal() + D * D)
        if mutation == "diagonal of B in fp16":
            E = half(E, sb)
        B = half(B - torch.diag(B.diagonal()), sb)
        V = E[:, None] * (hi.double() + lo.double()).float() + (B @ hi + B @ lo if rest else B @ hi)
    X = V.double() / S
    return X.t() if tall else X


def matrix(r, c, seed, rank=0, uneven=False, device="cpu"):
    """fp32 values: noise, or exactly ``rank`` directions up to fp32's own rounding; ``uneven``: rows of norms from 1
    to 2^-6."""
    g = torch.Generator().manual_seed(seed)
    if rank:
        G = torch.randn(r, rank, generator=g, dtype=torch.float64) @ torch.randn(rank, c, generator=g, dtype=torch.float64)
    else:
        G = torch.randn(r, c, generator=g, dtype=torch.float64)
    if uneven:
        G = G * torch.exp2(-6 * torch.rand(r, 1, generator=g, dtype=torch.float64))
    return G.float().to(device)


# (rows, columns, directions (0: all), uneven rows, steps) where each of MUTATIONS shows
CASES = [(64, 200, 16, False, 5), (50, 300, 2, True, 8), (96, 200, 4, False, 8), (300, 130, 4, True, 8), (256, 320, 16, False, 5),
         (600, 700, 16, False, 5), (600, 700, 4, True, 6), (900, 600, 0, True, 5)]


def case_matrix(case):
    r, c, rank, uneven, _ = case
    return matrix(r, c, 3, rank, uneven)


def share_of(got, G, steps, mutation):
    """How much of what ``mutation`` changes in the model ``got`` has (None: it changes nothing)."""
    like = rounded(G, steps)
    d = rounded(G, steps, mutation=mutation) - like
    size = float((d * d).sum())
    return float(((got - like) * d).sum()) / size if size else None


HEADER = """#include "ortho_plan.h"
extern "C" int scales(long r, int steps, float a, float b, float c, float *out) {
    const auto s = lce::ortho_plan::powers_of(r, steps, a, b, c);
    out[0] = s.x;
    out[1] = s.o;
    out[2] = s.b;
    return s.fit * 2 + s.rest;
}
extern "C" int shape(long batch, long rows_x, long rows_w, long steps) {
    return lce::ortho_plan::plan_of(batch, rows_x, rows_w, steps, false, false).shape;
}
"""


def load(directory: str):
    """(rows, steps, coefficients) -> (x, o, b, B X takes the rest), or None where they are refused, and (batch, rows,
    columns, rest) -> which tiles B X takes: the kernel's own choice, csrc/ortho_plan.h, compiled into ``directory``."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src, so = os.path.join(directory, "scales.cpp"), os.path.join(directory, "scales.so")
    with open(src, "w") as f:
        f.write(HEADER)
    csrc = os.path.join(root, "vocabulary_cross_entropy_row_amd", "csrc")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", f"-I{csrc}", src, "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.scales.argtypes = [ctypes.c_long, ctypes.c_int] + [ctypes.c_float] * 3 + [ctypes.c_void_p]

    def of(r, steps, abc):
        out = (ctypes.c_float * 3)()
        v = lib.scales(r, steps, *abc, ctypes.addressof(out))
        return (*out, bool(v & 1)) if v & 2 else None

    lib.shape.argtypes = [ctypes.c_long] * 4

    def shape(batch, rows, cols, rest):
        rp, cp = (-(-v // 64) * 64 for v in (min(rows, cols), max(rows, cols)))
        return lib.shape(batch, rp, cp, rp // 64 * (2 if rest else 1))

    return of, shape
