"""The paged 8-bit cache: quoka_cache_append, _select, _gather and _attn
against plain 64-bit forms, their edge cases, their refusals, and the calls
together as a serving loop makes them."""
import ctypes
import os
import subprocess
import sys
import threading

import pytest
import torch

from sparse_kv_selection_quoka_b200 import build
from tests import parity as P
from tests.test_library import _view, lib  # noqa: F401 (lib is a fixture)

E4M3 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
gpu = pytest.mark.gpu


def q():
    import sparse_kv_selection_quoka_b200 as m
    return m


# ------------------------------------------------------------ plain forms

def code_values():
    """The 256 values of e4m3, from the format: sign, 4 bits of exponent (bias 7), 3 of fraction."""
    out = []
    for u in range(256):
        e, f, s = (u >> 3) & 15, u & 7, -1.0 if u >> 7 else 1.0
        out.append(float("nan") if u & 127 == 127 else s * (f / 8 * 2.0**-6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)))
    return torch.tensor(out, dtype=torch.float64)


VALUES = code_values()
GRID = VALUES[:127]  # 0 .. 448, ascending


def encode(y):
    """e4m3 codes of 64-bit numbers: the nearest value, ties to the even code, at most 448 in magnitude."""
    m = y.abs().clamp(max=448.0).nan_to_num(0.0)
    hi = torch.searchsorted(GRID, m).clamp(max=126)  # GRID[hi] >= m
    lo = (hi - 1).clamp(min=0)
    up, down = GRID[hi] - m, m - GRID[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = torch.where(GRID[hi] == m, hi, code)
    code = code + 128 * torch.signbit(y).long()
    return torch.where(y.isnan(), 127, code).to(torch.uint8)


def same_codes(a, b):
    """Equal codes; the sign of a NaN is free."""
    nan = ((a & 127) == 127) & ((b & 127) == 127)
    return bool(((a == b) | nan).all())


class Pages:
    """A cache on the CPU: uint8 codes, scales, table and lengths, with the pages in random order."""

    def __init__(self, lens, room, nkv, d, page, seed, scales=(-3, 3), order="hnd"):
        g = torch.Generator().manual_seed(seed)
        self.page, self.nkv, self.d, self.lens = page, nkv, d, list(lens)
        b, cols = len(lens), max(1, -(-max(room) // page))
        need = [-(-r // page) for r in room]
        npages = sum(need) + 2
        ids = torch.randperm(npages, generator=g)
        self.table = torch.full((b, cols), 10**6, dtype=torch.int32)  # past the need: names no page
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = ids[at:at + n]
            at += n
        codes = torch.randint(0, 256, (2, npages, nkv, page, d), generator=g).to(torch.uint8)
        codes[(codes & 127) == 127] -= 1  # (NaN codes are planted where a test wants them)
        self.k, self.v = codes[0], codes[1]
        e = torch.randint(scales[0], scales[1] + 1, (2, npages, nkv), generator=g)
        self.k_scale, self.v_scale = (2.0 ** e[0]).float(), (2.0 ** e[1]).float()
        self.order = order

    def rows(self, i, n=None):
        """K, V (nkv, n, d) in 64 bits of sequence i."""
        n = self.lens[i] if n is None else n
        out = []
        for codes, scale in ((self.k, self.k_scale), (self.v, self.v_scale)):
            ids = self.table[i, : -(-n // self.page)].long()
            x = VALUES[codes[ids].long()] * scale[ids].double()[..., None, None]
            out.append(x.transpose(0, 1).reshape(self.nkv, len(ids) * self.page, self.d)[:, :n])
        return out

    def cuda(self, dtype=E4M3):
        def pool(c):
            if self.order == "nhd":  # rows of all heads next to one another
                return c.transpose(1, 2).contiguous().cuda().transpose(1, 2).view(dtype)
            return c.cuda().view(dtype)
        seq = torch.tensor(self.lens, dtype=torch.int32).cuda()
        return q().QuokaCache(pool(self.k), pool(self.v), self.k_scale.cuda(), self.v_scale.cuda(), self.table.cuda(), seq)


def rotate(x, cos, sin, neighbours):
    """x (h, t, d) fp32 by rows of cos, sin (t, rot / 2): elementary fp32 operations."""
    r = cos.shape[1]
    x = x.clone()
    if r:
        lo = slice(0, 2 * r, 2) if neighbours else slice(0, r)
        hi = slice(1, 2 * r, 2) if neighbours else slice(r, 2 * r)
        a, z = x[..., lo].clone(), x[..., hi].clone()
        x[..., lo] = a * cos - z * sin
        x[..., hi] = z * cos + a * sin
    return x


def append(c, K, V, cos, sin, neighbours, new):
    """Appends to the Pages c in place; returns the rotated keys (b, nkv, BCP, d) fp32."""
    turned = K.float().clone()
    for i, m in enumerate(new):
        n = c.lens[i]
        if m == 0:
            continue
        turned[i, :, :m] = rotate(K[i, :, :m].float(), cos[n:n + m], sin[n:n + m], neighbours)
        for codes, scales, x in ((c.k, c.k_scale, turned[i, :, :m]), (c.v, c.v_scale, V[i, :, :m].float())):
            for p in range(n // c.page, (n + m - 1) // c.page + 1):
                t0, t1, id_ = max(n, p * c.page), min(n + m, (p + 1) * c.page), int(c.table[i, p])
                for j in range(c.nkv):
                    y = x[j, t0 - n:t1 - n].double()
                    top = float(torch.where(y.isfinite(), y.abs(), 0.0).max())
                    e = -50
                    while e < 50 and top > 448 * 2.0**e:
                        e += 1
                    held = t0 - p * c.page
                    if held:
                        old = float(scales[id_, j])
                        e = max(e, round(torch.tensor(old).log2().item()))
                        codes[id_, j, :held] = encode(VALUES[codes[id_, j, :held].long()] * (old / 2.0**e))
                    scales[id_, j] = 2.0**e
                    codes[id_, j, held:held + t1 - t0] = encode(y * 2.0**-e)
    return turned


def attention(c, Q, Kc, Vc, idx=None, counts=None, scale=None):
    """O, lse in 64 bits, and what the error bounds are made of: per output
    sum_k p_k |v_k|, per row the largest sum_i |q_i k_i| * scale, and per output
    the sum over the cached keys of |v_k| 2^(E - ev_k), 2^ev_k a key's value
    scale and 2^E the largest."""
    b, nq, L, d = Q.shape
    G = nq // c.nkv
    scale = d**-0.5 if scale is None else scale
    O, A = torch.zeros(b, nq, L, d, dtype=torch.float64), torch.zeros(b, nq, L, d, dtype=torch.float64)
    B = torch.zeros_like(A)
    lse, size = torch.full((b, nq, L), -torch.inf, dtype=torch.float64), torch.zeros(b, nq, L, dtype=torch.float64)
    for i in range(b):
        K, V = c.rows(i)
        at_page = c.table[i, torch.arange(c.lens[i]) // c.page].long()
        for j in range(c.nkv):
            k, v, f = K[j], V[j], c.v_scale[at_page, j].double()
            if idx is not None:
                at = idx[i, j, : int(counts[i, j])].long()
                k, v, f = k[at], v[at], f[at]
            if f.numel():
                B[i, j * G:(j + 1) * G] = (v.abs() * (f.max() / f)[:, None]).sum(0)
            n = k.shape[0]
            if Kc is not None:
                k, v = torch.cat((k, Kc[i, j].double())), torch.cat((v, Vc[i, j].double()))
            for h in range(j * G, (j + 1) * G):
                for t in range(L):
                    m = n + (t + 1 if Kc is not None else 0)
                    if m == 0:
                        continue
                    x = Q[i, h, t].double()
                    s = (k[:m] @ x) * scale
                    lse[i, h, t] = torch.logsumexp(s, 0)
                    p = torch.exp(s - lse[i, h, t])
                    O[i, h, t], A[i, h, t] = p @ v[:m], p @ v[:m].abs()
                    size[i, h, t] = float((k[:m].abs() @ x.abs()).max()) * scale
    return O, lse, A, size, B


def check_attention(O, lse, want, dt, d, n, few):
    """Bounds on the kernels' roundings; few: at most 32 query rows per KV head,
    the codes' own kernel (fp32 always takes it).
    score: d fp32 additions of a tensor-core product, each off by at most
      2^-22 of the sum of magnitudes (`size`), and the fp32 query as two halves
      (2^-22): ds = (d + 8) 2^-22 size;
    weight: 2^x of an fp32 x, |x| <= 64 where it matters (2^-17), the rounding
      to the operand type (few rows, and fp32: fp16 2^-11, two halves 2^-21 for
      fp32 inputs; many bf16 rows: bf16 2^-8, and once more for a range's bf16
      partial), twice the score's error in numerator and denominator; with
      few rows 2^-32 of the largest w_k = p_k 2^ev_k at least (fp16 subnormals),
      which is at most 2^E L, L the denominator: 2^-32 B;
    sums: n keys, each addition off by 2^-22 of the sum of magnitudes;
    output: half a step of its type."""
    wO, wl, A, size, B = want
    ds = (d + 8) * 2.0**-22 * size
    few = few or dt == "f32"
    weight = {"bf16": 2.0**-11 if few else 2 * 2.0**-8, "f32": 2.0**-21}[dt]
    rel = weight + 2.0**-17 + 2 * ds + (n + 64) * 2.0**-22
    half = torch.finfo(TYPES[dt]).eps / 2
    O, lse = O.double().cpu(), lse.double().cpu()
    bad = (O - wO).abs() - (half * wO.abs() + 2 * rel[..., None] * A + (2.0**-32 * B if few else 0.0))
    assert O.isfinite().all() and bad.max() <= 0, f"O is {bad.max():.3e} past its bound"
    there = wl > -torch.inf
    assert torch.equal(lse > -torch.inf, there)
    off = (lse - wl)[there].abs() - (rel + 2.0**-22 * wl.abs())[there]
    assert off.numel() == 0 or off.max() <= 0, f"lse is {off.max():.3e} past its bound"


def randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def angles(npos, rot):
    a = torch.arange(npos, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(1, rot))
    return a.cos().float(), a.sin().float()


def strided(x):
    """x on the GPU as part of a larger tensor: other strides, the same values."""
    b, h, t, d = x.shape
    big = torch.full((b, t + 3, h + 1, d), float("nan"), dtype=x.dtype, device="cuda")
    view = big.transpose(1, 2)[:, :h, :t]
    view.copy_(x)
    return view


# ------------------------------------------------------------ append

APPENDS = [
    # lens, new (None: BCP each), BCP, nkv, nq, d, page, rot, neighbours, dtype, order of the pool
    ([0], None, 1, 1, 1, 64, 16, 64, False, "bf16", "hnd"),
    ([5, 63, 64, 127], None, 1, 2, 4, 128, 64, 128, False, "bf16", "hnd"),
    ([0, 15, 16, 30], [7, 0, 40, 39], 40, 3, 6, 64, 16, 32, True, "f32", "nhd"),
    ([100], None, 300, 2, 10, 128, 128, 64, False, "f32", "hnd"),
    ([31, 1], [200, 33], 200, 1, 8, 128, 32, 128, True, "bf16", "nhd"),
    ([17, 90], None, 129, 2, 2, 64, 128, 0, False, "bf16", "hnd"),
]


@gpu
@pytest.mark.parametrize("k", range(len(APPENDS)))
def test_append(k):
    """Codes, scales and the rotated copies, bit for bit; every byte of the
    pool that no new token concerns stays as it was."""
    lens, new, BCP, nkv, nq, d, page, rot, nb, dt, order = APPENDS[k]
    b, t = len(lens), TYPES[dt]
    c = Pages(lens, [n + BCP for n in lens], nkv, d, page, 10 + k, order=order)
    K, V, Q = randn(20 + k, b, nkv, BCP, d), randn(30 + k, b, nkv, BCP, d), randn(40 + k, b, nq, BCP, d)
    K *= torch.logspace(-3, 3, BCP)[:, None]  # pages whose scale has to grow, and ones where it need not
    V[:, :, ::5] = 0
    V[0, 0, 0, :3] = torch.tensor([float("inf"), -float("inf"), 1e30])
    K[0, 0, 0, 1] = float("inf") if rot == 0 else 3.0
    K, V, Q = K.to(t), V.to(t), Q.to(t)
    cos, sin = angles(max(lens) + BCP, rot)
    dev = c.cuda()
    nl = None if new is None else torch.tensor(new, dtype=torch.int32).cuda()
    Kr0, Qr0 = randn(1, *K.shape).to(t), randn(2, *Q.shape).to(t)
    Kr, Qr = Kr0.cuda(), Qr0.cuda()
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    got = q().quoka_cache_append(dev, strided(K), strided(V), strided(Q), *((cos.cuda(), sin.cuda()) if rot else (None, None)),
                                 interleaved=nb, new_len=nl, Kr=Kr, Qr=Qr, ws=ws)
    assert q().quoka_get_device_status(ws) == 0
    assert got[0] is Kr and got[1] is Qr
    news = [BCP] * b if new is None else new
    c2 = Pages(lens, [n + BCP for n in lens], nkv, d, page, 10 + k)
    turned = append(c2, K, V, cos, sin, nb, news)
    assert same_codes(dev.k.view(torch.uint8).cpu(), c2.k) and same_codes(dev.v.view(torch.uint8).cpu(), c2.v)
    assert torch.equal(dev.k_scale.cpu(), c2.k_scale) and torch.equal(dev.v_scale.cpu(), c2.v_scale)
    for i, m in enumerate(news):
        Kr0[i, :, :m] = turned[i, :, :m].to(t)
        Qr0[i, :, :m] = rotate(Q[i, :, :m].float(), cos[lens[i]:lens[i] + m], sin[lens[i]:lens[i] + m], nb).to(t)
    assert torch.equal(Kr.cpu().double(), Kr0.double()) and torch.equal(Qr.cpu().double(), Qr0.double())


@gpu
def test_append_special_values():
    """NaN stays NaN, infinities saturate, neither moves the scale; values
    beyond the scales' range saturate or vanish; codes with NaN are moved."""
    c = Pages([3], [64], 1, 64, 16, 5)
    c.k[c.table[0, 0].long(), 0, 1, 2] = 127
    K = torch.zeros(1, 1, 40, 64)
    K[0, 0, 0, 0], K[0, 0, 0, 1], K[0, 0, 1, 5] = float("nan"), -float("inf"), 1e4
    K[0, 0, 20] = 1e-30
    K[0, 0, 35, 3] = 3e38
    V = randn(3, 1, 1, 40, 64)
    dev = c.cuda(torch.uint8)
    q().quoka_cache_append(dev, K.cuda(), V.cuda())
    cos, sin = angles(64, 0)
    append(c, K, V, cos, sin, False, [40])
    assert same_codes(dev.k.cpu(), c.k) and same_codes(dev.v.cpu(), c.v)
    assert torch.equal(dev.k_scale.cpu(), c.k_scale) and torch.equal(dev.v_scale.cpu(), c.v_scale)


@gpu
def test_append_leaves_out_what_does_not_fit():
    """Positions past the table or the angles, bad counts and pages outside
    the cache are latched and left out; the rest is written."""
    c = Pages([60, 4, 10], [64, 40, 40], 1, 64, 16, 6)
    c.table[2, 1] = -5  # sequence 2's second page: tokens 16 .. 31
    K, V = randn(1, 3, 1, 20, 64), randn(2, 3, 1, 20, 64)
    dev = c.cuda(torch.uint8)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    q().quoka_cache_append(dev, K.cuda(), V.cuda(), new_len=torch.tensor([20, 20, 20], dtype=torch.int32).cuda(), ws=ws)
    assert q().quoka_get_device_status(ws) == 6
    cos, sin = angles(100, 0)
    lens = c.lens
    append(c, K, V, cos, sin, False, [4, 20, 6])
    assert same_codes(dev.k.cpu(), c.k) and torch.equal(dev.v_scale.cpu(), c.v_scale)
    # angles for 10 positions only: sequence 1 (4 held) takes 6 of its tokens, the others none
    c = Pages(lens, [64, 40, 40], 1, 64, 16, 6)
    dev = c.cuda(torch.uint8)
    cos, sin = angles(10, 64)
    q().quoka_cache_append(dev, K.cuda(), V.cuda(), None, cos.cuda(), sin.cuda(), ws=ws)
    assert q().quoka_get_device_status(ws) == 6
    append(c, K, V, cos, sin, False, [0, 6, 0])
    assert same_codes(dev.k.cpu(), c.k) and torch.equal(dev.k_scale.cpu(), c.k_scale)
    # a count outside [0, BCP], and a negative length
    c = Pages([4, 4, 4], [40, 40, 40], 1, 64, 16, 7)
    dev = c.cuda(torch.uint8)
    dev.seq_len[2] = -1
    q().quoka_cache_append(dev, K.cuda(), V.cuda(), new_len=torch.tensor([-3, 99, 5], dtype=torch.int32).cuda(), ws=ws)
    assert q().quoka_get_device_status(ws) == 6
    append(c, K, V, cos[:, :0], sin[:, :0], False, [0, 20, 0])
    assert same_codes(dev.k.cpu(), c.k) and same_codes(dev.v.cpu(), c.v)


@gpu
@pytest.mark.parametrize("dt,page,nq,BCP", [("bf16", 64, 9, 100), ("f32", 16, 3, 45), ("bf16", 128, 4, 1)])
def test_append_makes_zeros_of_what_is_left_out(dt, page, nq, BCP):
    """Rows of Kr and Qr made by the call: zeros for tokens past the page table, the
    angles or new_len and for all of a sequence whose length is none; the rotated
    rows for the rest. Rows of tensors that were given stay as they were."""
    m, t, d, nkv = q(), TYPES[dt], 64, 2
    cols = 3
    lens = [0, cols * page - 7, cols * page, -3, 10**9, cols * page - BCP]
    npos = cols * page - 2
    new = [BCP, BCP, 0, BCP, BCP, max(0, BCP - 3)]
    cos, sin = angles(npos, d)
    K, V, Q = (randn(s, len(lens), h, BCP, d).to(t) for s, h in ((1, nkv), (2, nkv), (3, nq)))
    for counts in (None, new):
        nl = None if counts is None else torch.tensor(counts, dtype=torch.int32).cuda()
        for given in ("", "Kr", "Qr"):
            dev = Pages([1] * 6, [cols * page] * 6, nkv, d, page, 5).cuda(torch.uint8)
            dev.seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
            kw = {"Kr": {"Kr": torch.full_like(K, 9.0).cuda()}, "Qr": {"Qr": torch.full_like(Q, 9.0).cuda()}}.get(given, {})
            up = K.cuda(), V.cuda(), Q.cuda(), cos.cuda(), sin.cuda()
            dirt = [torch.full(x.shape, float("nan"), dtype=t, device="cuda") for x in (K, Q)]
            del dirt  # (what the allocator hands out next)
            Kr, Qr = m.quoka_cache_append(dev, *up, new_len=nl, want_Kr=True, **kw)
            for i, n in enumerate(lens):
                fits = max(0, min(BCP, npos - n)) if 0 <= n <= npos else 0
                live = fits if counts is None else min(fits, counts[i])
                for name, got, x in (("Kr", Kr, K), ("Qr", Qr, Q)):
                    want = torch.full_like(x[i], 9.0 if name == given else 0.0)
                    if live:
                        want[:, :live] = rotate(x[i, :, :live].float(), cos[n:n + live], sin[n:n + live], False).to(t)
                    assert torch.equal(got[i].cpu(), want), (counts, given, i, name)


@gpu
def test_append_of_an_empty_chunk():
    c = Pages([5, 0], [20, 20], 2, 64, 16, 3)
    dev = c.cuda(torch.uint8)
    K, Q = torch.zeros(2, 2, 0, 64, device="cuda"), torch.zeros(2, 4, 0, 64, device="cuda")
    cos, sin = (x.cuda() for x in angles(20, 64))
    for kw in ({}, {"new_len": torch.zeros(2, dtype=torch.int32, device="cuda")}, {"Kr": torch.zeros_like(K)}):
        Kr, Qr = q().quoka_cache_append(dev, K, K, Q, cos, sin, want_Kr=True, **kw)
        assert Kr.shape == K.shape and Qr.shape == Q.shape
    assert torch.equal(dev.k.cpu(), c.k) and torch.equal(dev.k_scale.cpu(), c.k_scale)


@gpu
def test_append_of_no_tokens_needs_no_angles():
    """A sequence without new tokens may be longer than the table of angles."""
    c = Pages([30, 4], [64, 40], 1, 64, 16, 8)
    K, V = randn(1, 2, 1, 5, 64), randn(2, 2, 1, 5, 64)
    cos, sin = angles(10, 64)
    dev = c.cuda(torch.uint8)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    new = torch.tensor([0, 5], dtype=torch.int32).cuda()
    q().quoka_cache_append(dev, K.cuda(), V.cuda(), None, cos.cuda(), sin.cuda(), new_len=new, ws=ws)
    assert q().quoka_get_device_status(ws) == 0
    append(c, K, V, cos, sin, False, [0, 5])
    assert same_codes(dev.k.cpu(), c.k) and torch.equal(dev.k_scale.cpu(), c.k_scale)


# ------------------------------------------------------------ gather

GATHERS = [
    # lens, max_len, nkv, d, page, N (0: all rows), dtype, order
    ([1], 1, 1, 64, 16, 0, "bf16", "hnd"),
    ([77, 0, 200], 200, 2, 128, 64, 0, "f32", "nhd"),
    ([130, 129], 140, 3, 64, 128, 50, "bf16", "nhd"),
    ([1000, 3], 1000, 2, 128, 32, 333, "f32", "hnd"),
]


@gpu
@pytest.mark.parametrize("k", range(len(GATHERS)))
def test_gather(k):
    lens, max_len, nkv, d, page, N, dt, order = GATHERS[k]
    b = len(lens)
    c = Pages(lens, lens, nkv, d, page, 50 + k, scales=(-50, 50), order=order)
    c.k[c.table[0, 0].long(), 0, 0, 0] = 127
    idx = counts = None
    if N:
        g = torch.Generator().manual_seed(k)
        counts = torch.tensor([[min(n, N) if j == 0 else min(n, N) // 2 for j in range(nkv)] for n in lens], dtype=torch.int32)
        idx = torch.full((b, nkv, N), 2**31 - 1, dtype=torch.int32)
        for i, n in enumerate(lens):
            for j in range(nkv):
                m = int(counts[i, j])
                idx[i, j, :m] = torch.randint(0, n, (m,), generator=g)  # any order, repeats among them
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    K, V = q().quoka_cache_gather(c.cuda(), max_len, None if idx is None else idx.cuda(), None if idx is None else counts.cuda(),
                                  dtype=TYPES[dt], ws=ws)
    assert q().quoka_get_device_status(ws) == 0
    assert K.shape == (b, nkv, N or max_len, d) and K.dtype == TYPES[dt]
    for i, n in enumerate(lens):
        want = c.rows(i)
        for got, w in ((K[i], want[0]), (V[i], want[1])):
            for j in range(nkv):
                rows = w[j] if idx is None else w[j][idx[i, j, : int(counts[i, j])].long()]
                full = torch.zeros(N or max_len, d, dtype=torch.float64)
                full[: rows.shape[0]] = rows
                assert torch.equal(got[j].double().cpu().nan_to_num(12345.0), full.nan_to_num(12345.0))


# ------------------------------------------------------------ select

SELECTS = [
    # lens, max_len, nkv, nq, d, page, BCP, NQ, BSA, dtype, order
    ([1], 1, 1, 1, 64, 16, 1, 1, 1, "bf16", "hnd"),
    ([300, 0, 47, 129], 333, 2, 6, 128, 64, 20, 3, 50, "bf16", "nhd"),
    ([999], 1000, 3, 3, 64, 16, 70, 70, 1000, "f32", "hnd"),
    ([2500, 1], 5001, 2, 16, 128, 32, 64, 17, 600, "f32", "hnd"),
    ([6000, 5999], 6000, 2, 8, 128, 128, 1, 1, 512, "bf16", "hnd"),
    ([20000], 20000, 1, 4, 64, 64, 33, 8, 4000, "bf16", "hnd"),
    ([(71 * i) % 311 for i in range(50)], 310, 3, 3, 128, 16, 1, 1, 40, "bf16", "hnd"),  # 150 rows, ragged
    ([513, 512], 1025, 1, 5, 64, 16, 9, 5, 100, "bf16", "nhd"),
    ([300] * 5 + [7] * 12, 300, 2, 8, 128, 32, 12, 3, 30, "bf16", "hnd"),  # more query heads than SMs
    ([1500, 130, 0], 1500, 2, 4, 128, 64, 90, 24, 200, "bf16", "nhd"),    # group means in full groups of pieces
    ([1400, 1], 1400, 1, 2, 64, 32, 90, 25, 200, "f32", "hnd"),           # the coarser pieces
    ([260], 260, 2, 2, 128, 128, 200, 130, 60, "f32", "nhd"),             # five passes
]


def select_oracle(c, Q, q_idx):
    """S_agg (b, nkv, L) in 64 bits for the chosen positions q_idx, by the definition."""
    b, nq, _, d = Q.shape
    unit = Q.double() / Q.double().norm(dim=-1, keepdim=True)
    picked = unit.gather(2, q_idx.long()[..., None].expand(-1, -1, -1, d))
    group = picked.view(b, c.nkv, nq // c.nkv, -1, d).mean(2)
    out = []
    for i in range(b):
        K = c.rows(i)[0]
        n = K.norm(dim=-1, keepdim=True)
        K = torch.where(n > 0, K / n.clamp(min=1e-300), 0.0)
        out.append((K @ group[i].transpose(1, 2)).amax(-1))
    return out


@gpu
@pytest.mark.parametrize("k", range(len(SELECTS)))
def test_select(k):
    """The scores' bound: the group mean of unit queries (d additions and a
    square root, (d + 8) 2^-24), its two halves (2^-22; more than four of them:
    pieces, 2^-20, more than 24: 2^-16), d additions of the product and d of
    |k|^2 (each 2^-22 of magnitudes that Cauchy bounds by 1): (2 d + 16) 2^-22,
    and 2^-16 with the coarser pieces. Keys may swap across the last place
    within twice that."""
    lens, max_len, nkv, nq, d, page, BCP, NQ, BSA, dt, order = SELECTS[k]
    b, n = len(lens), min(BSA, max_len)
    c = Pages(lens, [max_len] + lens[1:], nkv, d, page, 60 + k, scales=(-50, 50), order=order)
    c.k[c.table[0, 0].long(), 0, 0] = 0  # a key of zeros: scores 0
    Q = (randn(70 + k, b, nq, BCP, d) + 1.0).to(TYPES[dt])
    kv_idx = torch.full((b, nkv, n), -7, dtype=torch.int32, device="cuda")
    s_agg = torch.full((b, nkv, max_len), 5.0, device="cuda")
    size = q().quoka_select_workspace_size(b, nq, nkv, d, max_len, BCP, NQ, BSA, TYPES[dt])
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    idx, count, q_idx, s = q().quoka_cache_select(strided(Q), c.cuda(), max_len, NQ, BSA, kv_idx=kv_idx, s_agg=s_agg,
                                                  want_q_idx=True, ws=ws)
    assert q().quoka_get_device_status(ws) == 0
    # the chosen queries: rank order of -cos(Q, mean), near-ties may swap
    mean = Q.double().mean(2, keepdim=True)
    SQ = -torch.nn.functional.cosine_similarity(Q.double(), mean, dim=-1, eps=1e-300)
    want_q = SQ.sort(dim=-1, descending=True, stable=True).indices[..., :NQ]
    P.check_q_idx(q_idx.cpu().numpy(), SQ.numpy(), want_q.numpy())
    want = select_oracle(c, Q, q_idx.cpu())
    tol = (2 * d + 16) * 2.0**-22 + (2.0**-16 if NQ > 24 else 0.0)
    for i, L in enumerate(lens):
        m = min(n, L)
        got = s[i].double().cpu()
        assert (got[:, :L] - want[i]).abs().max() <= tol if L else True
        assert (got[:, L:] == 5.0).all() and (idx[i, :, m:] == -7).all() and (count[i] == m).all()
        for j in range(nkv):
            # the picks are exactly the best of the scores returned, ties to the lower index ...
            best = got[j, :L].sort(descending=True, stable=True).indices[:m].sort().values
            assert torch.equal(idx[i, j, :m].cpu().long(), best)
            # ... and of the true ones up to their bound
            if m:
                last = want[i][j].sort(descending=True).values[m - 1]
                assert (want[i][j][best] >= last - 2 * tol).all()


@gpu
@pytest.mark.parametrize("NQ", [5, 24, 25, 49, 130])
def test_select_scores_to_the_last_piece(NQ):
    """Half of a key's columns are 1, the rest 0; a query is 1 there and beta
    elsewhere, so that its unit vector has any fraction beta gives it (these leave
    the most behind four pieces), products and their sums are exact, and the score
    is sqrt(m / (m + (d - m) beta^2)). Bound, relative: five pieces 2^-24, four (more
    than 24 group means) 2^-19, rsqrt 2^-22, and 2^-24 for each of: 34 additions of
    |q|^2, halved by the root, the root, the division, four joins of pieces, two
    products."""
    d, m, BCP = 128, 64, max(NQ, 40)
    beta = [1.39988, 1.30399, 1.3056, 1.35226, 0.98057, 1.18919, 1.12156, 1.39372, 1.32614, 0.50759, 0.60337, 0.66868, 0.80136,
            0.93802, 0.29239, 0.64385]
    c = Pages([30] * 16, [30] * 16, 1, d, 16, 5)
    c.k[:] = 0
    c.k[..., ::2] = 56  # 1.0
    Q = torch.ones(16, 1, BCP, d)
    Q[..., 1::2] = torch.tensor(beta)[:, None, None, None]
    _, _, _, s = q().quoka_cache_select(Q.cuda(), c.cuda(), 30, NQ, 4, want_s_agg=True)
    b, piece = torch.tensor(beta).double(), 2.0 ** (-24 if NQ <= 24 else -19)  # (beta as fp32 holds it)
    want = (m / (m + (d - m) * b * b)).sqrt()[:, None].expand(16, 30)
    assert ((s[:, 0].double().cpu() / want - 1).abs() <= piece + 2.0**-22 + 25 * 2.0**-24).all()


PADDED = [
    # lens, new, nkv, nq, d, page, BCP, NQ, BSA, dtype, what the rows of padding hold
    ([300, 47, 129, 200], [33, 1, 0, 100], 2, 8, 128, 64, 100, 4, 50, "bf16", 0.0),
    ([300, 47, 129, 200], [33, 1, 0, 100], 2, 8, 128, 64, 100, 4, 50, "bf16", float("nan")),
    ([90, 31, 0, 77], [1, 0, 1, 1], 2, 6, 128, 32, 1, 1, 20, "bf16", float("nan")),
    ([500, 400, 300, 10], [129, 20, 3, 200], 1, 3, 64, 16, 200, 30, 64, "f32", 0.0),     # a cluster a head
    ([260, 250], [3990, 2], 1, 2, 128, 128, 4000, 5, 40, "f32", float("inf")),          # rows from global memory
    ([1500, 130, 64], [90, 16, 5], 2, 4, 128, 64, 90, 17, 200, "bf16", -30.0),          # group means in pieces
    ([3000, 2500, 2900], [0, 7, 12], 2, 4, 64, 32, 12, 3, 600, "bf16", 0.0),            # the larger top-k
    ([70000, 66000], [3, 0], 1, 1, 64, 128, 5, 2, 300, "f32", 1e30),                    # the largest
]


@gpu
@pytest.mark.parametrize("k", range(len(PADDED)))
def test_select_of_a_padded_chunk(k):
    """Rows behind new_len are no queries, whatever they hold: the choice is that
    of the sequence's own chunk, the scores those of the chosen (the bounds of
    test_select), and a sequence without queries selects nothing."""
    lens, new, nkv, nq, d, page, BCP, NQ, BSA, dt, fill = PADDED[k]
    b, max_len = len(lens), max(lens)
    c = Pages(lens, lens, nkv, d, page, 160 + k)
    Q = (randn(170 + k, b, nq, BCP, d) + 1.0).to(TYPES[dt])
    for i, m in enumerate(new):
        Q[i, :, m:] = fill
    kv_idx = torch.full((b, nkv, min(BSA, max_len)), -7, dtype=torch.int32, device="cuda")
    s_agg = torch.full((b, nkv, max_len), 5.0, device="cuda")
    size = q().quoka_select_workspace_size(b, nq, nkv, d, max_len, BCP, NQ, BSA, TYPES[dt])
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    idx, count, q_idx, s = q().quoka_cache_select(Q.cuda(), c.cuda(), max_len, NQ, BSA, kv_idx=kv_idx, s_agg=s_agg, ws=ws,
                                                  new_len=torch.tensor(new, dtype=torch.int32).cuda(), want_q_idx=True)
    assert q().quoka_get_device_status(ws) == 0
    tol = (2 * d + 16) * 2.0**-22 + (2.0**-16 if NQ > 24 else 0.0)
    for i, (L, m) in enumerate(zip(lens, new)):
        take = min(BSA, L) if m else 0
        assert (count[i] == take).all() and (idx[i, :, take:] == -7).all()
        keep = min(NQ, m)
        assert (q_idx[i, :, keep:] == -1).all()
        if m == 0:
            assert (s[i] == 5.0).all()
            continue
        own = Q[i:i + 1, :, :m]
        SQ = -torch.nn.functional.cosine_similarity(own.double(), own.double().mean(2, keepdim=True), dim=-1, eps=1e-300)
        at = q_idx[i:i + 1, :, :keep].cpu()
        P.check_q_idx(at.numpy(), SQ.numpy(), SQ.sort(dim=-1, descending=True, stable=True).indices[..., :keep].numpy())
        one = Pages.__new__(Pages)
        one.__dict__.update(c.__dict__, table=c.table[i:i + 1], lens=lens[i:i + 1])
        want = select_oracle(one, own, at)[0]
        got = s[i].double().cpu()
        assert (got[:, :L] - want).abs().max() <= tol if L else True
        assert (got[:, L:] == 5.0).all()
        for j in range(nkv):
            best = got[j, :L].sort(descending=True, stable=True).indices[:take].sort().values
            assert torch.equal(idx[i, j, :take].cpu().long(), best)


@gpu
def test_padded_chunk_in_a_graph_and_out_of_range():
    """A captured selection follows new_len; a count that is none latches."""
    m, b, BCP = q(), 3, 70
    c = Pages([400, 300, 350], [400, 300, 350], 2, 128, 32, 9).cuda()
    Q = randn(8, b, 4, BCP, 128).to(torch.bfloat16).cuda()
    new = torch.tensor([70, 70, 70], dtype=torch.int32).cuda()
    ws = torch.zeros(m.quoka_select_workspace_size(b, 4, 2, 128, 400, BCP, 4, 50, Q.dtype), dtype=torch.uint8, device="cuda")
    idx, cnt = torch.zeros(b, 2, 50, dtype=torch.int32, device="cuda"), torch.zeros(b, 2, dtype=torch.int32, device="cuda")
    call = lambda: m.quoka_cache_select(Q, c, 400, 4, 50, new_len=new, kv_idx=idx, kv_count=cnt, ws=ws)
    call()
    plain, _, _, _ = m.quoka_cache_select(Q, c, 400, 4, 50)
    assert torch.equal(idx, plain)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for counts in ([70, 5, 0], [1, 69, 33]):
        new.copy_(torch.tensor(counts, dtype=torch.int32))
        Q.normal_()
        idx.fill_(-7)
        g.replay()
        got = idx.clone(), cnt.clone()
        idx.fill_(-7)
        call()
        assert torch.equal(got[0], idx) and torch.equal(got[1], cnt) and m.quoka_get_device_status(ws) == 0
        assert cnt.tolist() == [[50 if n else 0] * 2 for n in counts]
    for counts in ([71, 5, 5], [5, 5, -1]):
        new.copy_(torch.tensor(counts, dtype=torch.int32))
        call()
        assert m.quoka_get_device_status(ws) == 6 and (cnt == 0).all()


@gpu
def test_select_ties_go_to_the_lower_index():
    c = Pages([400], [400], 1, 128, 32, 3)
    for t in range(400):  # ten kinds of keys, in scales that do not matter
        p, r = divmod(t, 32)
        c.k[int(c.table[0, p]), 0, r] = c.k[int(c.table[0, 0]), 0, t % 10]
    Q = randn(4, 1, 4, 8, 128).to(torch.bfloat16)
    idx, count, _, s = q().quoka_cache_select(Q.cuda(), c.cuda(), 400, 2, 100, want_s_agg=True)
    s = s[0, 0].cpu()
    assert torch.equal(s[:10].repeat(40), s)
    assert torch.equal(idx[0, 0].cpu().long(), s.sort(descending=True, stable=True).indices[:100].sort().values)


# ------------------------------------------------------------ attention

ATTNS = [
    # lens, max_len, nkv, nq, d, page, BCP, N (0: all keys), chunk keys, dtype, order
    ([1], 1, 1, 1, 64, 16, 1, 0, False, "bf16", "hnd"),
    ([0, 300, 17, 64], 300, 2, 8, 128, 64, 1, 0, True, "bf16", "nhd"),
    ([0, 299, 16], 300, 2, 6, 64, 16, 1, 0, False, "f32", "hnd"),
    ([700, 9], 700, 1, 7, 128, 32, 5, 0, True, "f32", "hnd"),
    ([900], 1000, 2, 16, 128, 128, 8, 333, True, "bf16", "nhd"),
    ([500, 40], 500, 3, 6, 64, 64, 3, 100, False, "f32", "hnd"),
    ([0, 260], 260, 1, 5, 128, 16, 13, 0, True, "bf16", "hnd"),      # 65 rows: the dense path
    ([300, 0], 310, 2, 4, 128, 64, 130, 200, True, "bf16", "hnd"),
    ([150], 150, 1, 3, 64, 16, 70, 0, True, "bf16", "nhd"),
    ([90, 200], 200, 1, 8, 64, 32, 16, 77, False, "f32", "hnd"),
    ([0], 0, 1, 2, 128, 16, 40, 0, True, "bf16", "hnd"),             # no cached key at all
    ([0], 0, 1, 2, 64, 16, 2, 0, True, "f32", "hnd"),
    ([20000], 20000, 1, 2, 128, 128, 1, 0, False, "bf16", "hnd"),    # one row in more ranges than are fetched ahead
    ([5000, 4900, 0], 5000, 1, 10, 64, 64, 5, 0, True, "f32", "nhd"),  # the same, with the rows of a full GPU
    ([(37 * i) % 131 for i in range(40)], 128, 2, 4, 64, 32, 1, 0, False, "bf16", "hnd"),  # 80 rows, ragged
    ([(29 * i) % 23 for i in range(150)], 22, 4, 4, 64, 16, 1, 7, True, "f32", "nhd"),     # 600 rows, tiny
    ([200], 200, 1, 2, 64, 16, 170, 50, True, "f32", "hnd"),         # fp32 in six blocks of rows
    ([900, 31], 1000, 2, 4, 64, 128, 150, 0, False, "bf16", "nhd"),   # d = 64 on the dense path, split key ranges
    ([700], 700, 1, 1, 64, 32, 257, 129, True, "bf16", "hnd"),
]


def index_lists(lens, nkv, N, seed):
    g = torch.Generator().manual_seed(seed)
    counts = torch.tensor([[min(n, N) if j == 0 else min(n, N) // 3 for j in range(nkv)] for n in lens], dtype=torch.int32)
    idx = torch.full((len(lens), nkv, N), 2**31 - 1, dtype=torch.int32)
    for i, n in enumerate(lens):
        for j in range(nkv):
            m = int(counts[i, j])
            idx[i, j, :m] = torch.randperm(max(1, n), generator=g)[:m].sort().values
    return idx, counts


@gpu
@pytest.mark.parametrize("k", range(len(ATTNS)))
def test_attention(k):
    lens, max_len, nkv, nq, d, page, BCP, N, chunk, dt, order = ATTNS[k]
    b, t = len(lens), TYPES[dt]
    c = Pages(lens, lens, nkv, d, page, 80 + k, scales=(-9, -5), order=order)
    # what lies behind a sequence's end in its last page must not matter
    for i, n in enumerate(lens):
        if n % page:
            p = int(c.table[i, n // page])
            c.k[p, :, n % page:] = 127
            c.v[p, :, n % page:] = 127
    idx = counts = None
    if N:
        idx, counts = index_lists(lens, nkv, N, k)
    Q = (2 * randn(90 + k, b, nq, BCP, d)).to(t)
    Kc, Vc = (randn(s + k, b, nkv, BCP, d).to(t) for s in (100, 110)) if chunk else (None, None)
    size = q().quoka_cache_attn_workspace_size(b, nq, nkv, d, BCP, N or max_len, t)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    up = lambda x: None if x is None else x.cuda()
    O, lse = q().quoka_cache_attn(strided(Q), c.cuda(), max_len, up(idx), up(counts), None if Kc is None else strided(Kc),
                                  None if Vc is None else strided(Vc), want_lse=True, ws=ws)
    assert q().quoka_get_device_status(ws) == 0
    check_attention(O, lse, attention(c, Q, Kc, Vc, idx, counts), dt, d, (N or max_len) + BCP, nq // nkv * BCP <= 32)


PACKED = [
    # lens, max_len, nkv, nq, d, page, BCP, N (0: all keys), chunk keys: contiguous Q, several heads a tile
    ([300, 0], 300, 1, 4, 128, 64, 200, 0, True),       # seven tiles, two of chunk keys; tiles that begin in another head
    ([300, 17], 304, 1, 4, 64, 16, 200, 90, True),
    ([6000, 130, 0], 6000, 1, 3, 128, 128, 70, 0, True),  # two tiles in sixteen ranges, most of them empty of the short rows
    ([6000, 1], 6000, 1, 3, 64, 32, 70, 0, False),
    ([5000, 4000], 5000, 2, 6, 64, 64, 50, 1900, True),
    ([2100], 2100, 2, 80, 128, 32, 1, 0, True),          # a decode step of forty heads a KV head
    ([700], 700, 1, 8, 128, 16, 130, 0, False),
]


@gpu
@pytest.mark.parametrize("k", range(len(PACKED)))
def test_attention_of_packed_heads(k):
    """Chunks of many bf16 rows whose heads follow one another without a gap: a tile
    takes rows of several heads. Against the plain form, and, but for the ranges'
    rounding, what a Q of other strides gives."""
    lens, max_len, nkv, nq, d, page, BCP, N, chunk = PACKED[k]
    b, t = len(lens), torch.bfloat16
    G = nq // nkv
    assert G * BCP > 32 and nkv * -(-G * BCP // 128) < nq * -(-BCP // 128)
    c = Pages(lens, lens, nkv, d, page, 180 + k, scales=(-9, -5))
    for i, n in enumerate(lens):
        if n % page:
            p = int(c.table[i, n // page])
            c.k[p, :, n % page:] = 127
            c.v[p, :, n % page:] = 127
    idx, counts = index_lists(lens, nkv, N, k) if N else (None, None)
    Q = (2 * randn(190 + k, b, nq, BCP, d)).to(t)
    Kc, Vc = (randn(s + k, b, nkv, BCP, d).to(t) for s in (200, 210)) if chunk else (None, None)
    size = q().quoka_cache_attn_workspace_size(b, nq, nkv, d, BCP, N or max_len, t)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    up = lambda x: None if x is None else x.cuda()
    dev, want = c.cuda(), attention(c, Q, Kc, Vc, idx, counts)
    for rows in (Q.cuda(), strided(Q)):
        O, lse = q().quoka_cache_attn(rows, dev, max_len, up(idx), up(counts), up(Kc), up(Vc), want_lse=True, ws=ws)
        assert q().quoka_get_device_status(ws) == 0
        check_attention(O, lse, want, "bf16", d, (N or max_len) + BCP, False)


@gpu
@pytest.mark.parametrize("dt,d,BCP,nq,N", [("bf16", 128, 1, 8, 0), ("bf16", 128, 40, 4, 0), ("bf16", 64, 40, 4, 50),
                                           ("f32", 64, 9, 4, 0), ("bf16", 128, 1, 70, 0)])
def test_attention_of_broadcast_rows(dt, d, BCP, nq, N):
    """Queries and chunk rows that several sequences and heads share by a stride
    of 0, and a single query row between others (its row stride says nothing)."""
    c = Pages([130, 77], [130, 77], 2 if nq < 70 else 1, d, 32, 12, scales=(-9, -5))
    t, nkv = TYPES[dt], c.nkv
    idx = counts = None
    if N:
        idx, counts = index_lists([130, 77], nkv, N, 3)
    Q, K, V = (randn(s, 1, 1, BCP, d).to(t).cuda() for s in (1, 2, 3))
    if BCP == 1:  # (b, 1, nq, d) seen as (b, nq, 1, d)
        Q = randn(1, 2, 1, nq, d).to(t).cuda().transpose(1, 2)
    else:
        Q = Q.expand(2, nq, BCP, d)
    K, V = K.expand(2, nkv, BCP, d), V.expand(2, nkv, BCP, d)
    up = lambda x: None if x is None else x.cuda()
    O, lse = q().quoka_cache_attn(Q, c.cuda(), 130, up(idx), up(counts), K, V, want_lse=True)
    want = attention(c, Q.cpu(), K.cpu(), V.cpu(), idx, counts)
    check_attention(O, lse, want, dt, d, (N or 130) + BCP, nq // nkv * BCP <= 32)


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_attention_far_scales_and_scores(dt):
    """Pages whose scales lie far apart: the largest scores in pages of tiny
    values and the largest values under tiny scores, in ascending order of
    both, so that the running maximum moves all the time; a large softmax
    scale leaves one key."""
    c = Pages([640], [640], 1, 64, 16, 9, scales=(-9, -7))
    for p in range(40):
        id_ = int(c.table[0, p])
        c.v_scale[id_, 0] = 2.0 ** (50 - (p * 5) % 101)
        c.k_scale[id_, 0] = 2.0 ** (-12 + p // 8)
    Q = randn(1, 1, 3, 1, 64).to(TYPES[dt])
    for scale in (0.05, 0.4):
        O, lse = q().quoka_cache_attn(Q.cuda(), c.cuda(), 640, scale=scale, want_lse=True)
        want = attention(c, Q, None, None, scale=scale)
        check_attention(O, lse, want, dt, 64, 640, True)


@gpu
def test_attention_nan_reaches_its_rows_only():
    """A NaN or an infinity among the inputs makes NaN of the rows that see
    it and of no others."""
    c = Pages([100, 100], [100, 100], 2, 64, 16, 4, scales=(-8, -6))
    c.k[int(c.table[0, 3]), 1, 2, 7] = 127
    Q = randn(1, 2, 4, 1, 64)
    Q[1, 0, 0, 5] = float("inf")
    O, _ = q().quoka_cache_attn(Q.cuda(), c.cuda(), 100)
    nan = O.isnan().all(-1)[..., 0].cpu()
    assert torch.equal(nan, torch.tensor([[False, False, True, True], [True, False, False, False]]))
    assert torch.equal(O.isnan().any(-1)[..., 0].cpu(), nan)


# ------------------------------------------------------------ device faults

@gpu
def test_reads_latch_what_is_out_of_range():
    """A bad page reads as zeros, a bad index as a zero row, a length beyond
    max_len as max_len; each is latched, and the next good call clears it."""
    c = Pages([100], [100], 1, 64, 16, 8, scales=(-8, -6))
    Q, good = randn(1, 1, 2, 1, 64), c.cuda()
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    status = lambda: q().quoka_get_device_status(ws)

    def calls(cache, max_len=100, idx=None):
        cnt = None if idx is None else torch.tensor([[idx.shape[2]]], dtype=torch.int32).cuda()
        K, _ = q().quoka_cache_gather(cache, max_len, idx, cnt, dtype=torch.float32, ws=ws)
        seen = [status()]
        O, _ = q().quoka_cache_attn(Q.cuda(), cache, max_len, idx, cnt, ws=ws)
        seen.append(status())
        if idx is None:
            q().quoka_cache_select(Q.cuda(), cache, max_len, 1, 5, ws=ws)
            seen.append(status())
        return seen, K, O

    table = c.table.clone()
    c.table[0, 2] = 10**6
    seen, K, O = calls(c.cuda())
    assert seen == [6, 6, 6] and (K[0, 0, 32:48] == 0).all() and K[0, 0, :32].abs().sum() > 0 and O.isfinite().all()
    c.table = table
    assert calls(good)[0] == [0, 0, 0]
    seen, K, O = calls(good, max_len=50)
    assert seen == [6, 6, 6] and torch.equal(K, calls(good)[1][:, :, :50])
    seen, K, O = calls(good, idx=torch.tensor([[[3, -1, 100, 99]]], dtype=torch.int32).cuda())
    assert seen == [6, 6] and (K[0, 0, 1:3] == 0).all() and O.isfinite().all()
    c.k_scale[c.table[0, 1].long()] = 0.3  # not a power of two
    assert calls(c.cuda())[0][:2] == [6, 6]


# ------------------------------------------------------------ the calls together

@gpu
@pytest.mark.parametrize("dt,d", [("bf16", 128), ("f32", 64)])
def test_serving_loop(dt, d):
    """Two ragged prompts taken in by chunks and continued token by token:
    append with rotation, select, attend over the selection and the chunk,
    advance. The cache of every step is the plain one bit for bit; the
    attention is checked on the selection made."""
    t, nkv, nq, page, NQ, BSA = TYPES[dt], 2, 6, 16, 4, 24
    c = Pages([0, 0], [160, 160], nkv, d, page, 11)
    dev, room = c.cuda(torch.uint8), 160
    cos, sin = angles(room, d)
    steps = [(40, [40, 33]), (40, [40, 1]), (40, [20, 0])] + [(1, [1, 1])] * 4 + [(5, [5, 3])]
    for k, (BCP, new) in enumerate(steps):
        K, V, Q = (randn(200 + 3 * k + u, 2, h, BCP, d).to(t) for u, h in enumerate((nkv, nkv, nq)))
        nl = torch.tensor(new, dtype=torch.int32).cuda()
        Kr, Qr = q().quoka_cache_append(dev, K.cuda(), V.cuda(), Q.cuda(), cos.cuda(), sin.cuda(), new_len=nl, want_Kr=True)
        max_len = max(1, max(c.lens))
        idx, cnt, _, _ = q().quoka_cache_select(Qr, dev, max_len, min(NQ, BCP), BSA)
        O, lse = q().quoka_cache_attn(Qr, dev, max_len, idx, cnt, Kr, V.cuda(), want_lse=True)
        want = attention(c, Qr.cpu(), Kr.cpu(), V, idx.cpu(), cnt.cpu())
        for i, m in enumerate(new):  # rows of padded tokens are nobody's
            check_attention(O[i:i + 1, :, :m], lse[i:i + 1, :, :m], [w[i:i + 1, :, :m] for w in want], dt, d,
                            idx.shape[2] + BCP, nq // nkv * BCP <= 32) if m else None
        append(c, K, V, cos, sin, False, new)
        assert same_codes(dev.k.cpu(), c.k) and same_codes(dev.v.cpu(), c.v)
        assert torch.equal(dev.k_scale.cpu(), c.k_scale) and torch.equal(dev.v_scale.cpu(), c.v_scale)
        dev.seq_len += nl
        c.lens = [n + m for n, m in zip(c.lens, new)]


@gpu
@pytest.mark.parametrize("dt,d", [("bf16", 128), ("f32", 64)])
def test_serving_loop_selects_for_its_own_tokens(dt, d):
    """Padded chunks through append, select and attention: every sequence's
    selection is that of its own tokens alone, by the definition in 64 bits (the
    scores' bound of test_select)."""
    t, nkv, nq, page, NQ, BSA = TYPES[dt], 2, 6, 16, 4, 24
    c = Pages([0, 0, 0], [160, 160, 160], nkv, d, page, 12)
    dev = c.cuda(torch.uint8)
    cos, sin = angles(160, d)
    for k, (BCP, new) in enumerate([(70, [70, 41, 0]), (40, [33, 40, 1]), (40, [2, 0, 40]), (1, [1, 0, 1]), (5, [5, 3, 1])]):
        K, V, Q = (randn(300 + 3 * k + u, 3, h, BCP, d).to(t) for u, h in enumerate((nkv, nkv, nq)))
        nl = torch.tensor(new, dtype=torch.int32).cuda()
        Kr, Qr = q().quoka_cache_append(dev, K.cuda(), V.cuda(), Q.cuda(), cos.cuda(), sin.cuda(), new_len=nl, want_Kr=True)
        max_len = max(1, max(c.lens))
        n = min(NQ, BCP)
        idx, cnt, at, _ = q().quoka_cache_select(Qr, dev, max_len, n, BSA, new_len=nl, want_q_idx=True)
        O, lse = q().quoka_cache_attn(Qr, dev, max_len, idx, cnt, Kr, V.cuda(), want_lse=True)
        want = attention(c, Qr.cpu(), Kr.cpu(), V, idx.cpu(), cnt.cpu())
        tol = (2 * d + 16) * 2.0**-22
        for i, m in enumerate(new):
            take = min(BSA, c.lens[i]) if m else 0
            assert (cnt[i] == take).all()
            if m == 0:
                continue
            own, keep = Qr[i:i + 1, :, :m].cpu(), min(n, m)
            assert ((at[i, :, :keep] >= 0) & (at[i, :, :keep] < m)).all() and (at[i, :, keep:] == -1).all()
            SQ = -torch.nn.functional.cosine_similarity(own.double(), own.double().mean(2, keepdim=True), dim=-1, eps=1e-300)
            P.check_q_idx(at[i:i + 1, :, :keep].cpu().numpy(), SQ.numpy(),
                          SQ.sort(dim=-1, descending=True, stable=True).indices[..., :keep].numpy())
            one = Pages.__new__(Pages)
            one.__dict__.update(c.__dict__, table=c.table[i:i + 1], lens=c.lens[i:i + 1])
            true = select_oracle(one, own, at[i:i + 1, :, :keep].cpu())[0]
            for j in range(nkv):
                pick = idx[i, j, :take].cpu().long()
                assert len(set(pick.tolist())) == take
                if take:
                    assert (true[j][pick] >= true[j].sort(descending=True).values[take - 1] - 2 * tol).all()
            check_attention(O[i:i + 1, :, :m], lse[i:i + 1, :, :m], [w[i:i + 1, :, :m] for w in want], dt, d,
                            idx.shape[2] + BCP, nq // nkv * BCP <= 32)
        append(c, K, V, cos, sin, False, new)
        dev.seq_len += nl
        c.lens = [n_ + m for n_, m in zip(c.lens, new)]


@gpu
def test_decode_step_replays_from_a_cuda_graph():
    """A captured decode step follows the lengths, tables and inputs it finds
    at each replay, on another stream too; two captured graphs with workspaces
    of their own do not disturb one another."""
    m, t = q(), torch.bfloat16
    c = Pages([30, 50], [128, 128], 2, 128, 16, 12)
    dev = c.cuda(torch.uint8)
    cos, sin = (x.cuda() for x in angles(128, 128))
    K, V = (torch.zeros(2, 2, 1, 128, dtype=t, device="cuda") for _ in range(2))
    Q = torch.zeros(2, 8, 1, 128, dtype=t, device="cuda")

    def step():
        Kr, Qr = m.quoka_cache_append(dev, K, V, Q, cos, sin, want_Kr=True)
        idx, cnt, _, _ = m.quoka_cache_select(Qr, dev, 128, 1, 20)
        O, lse = m.quoka_cache_attn(Qr, dev, 128, idx, cnt, Kr, V, want_lse=True)
        full, _ = m.quoka_cache_attn(Qr, dev, 128, None, None, Kr, V)
        return Kr, Qr, cnt, O, lse, full

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    state = [x.clone() for x in (dev.k, dev.v, dev.k_scale, dev.v_scale)]
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    for k in range(3):
        for x, u in ((K, 0), (V, 1), (Q, 2)):
            x.copy_(randn(300 + 3 * k + u, *x.shape).to(t))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for g in graphs:  # the same step twice: append writes the same tokens again
                g.replay()
        side.synchronize()
        got = [x.clone() for x in outs[0]]
        assert all(torch.equal(x, y) for x, y in zip(got, outs[1]))
        for x, y in zip((dev.k, dev.v, dev.k_scale, dev.v_scale), state):
            x.copy_(y)
        assert all(torch.equal(x, y) for x, y in zip(got, step()))
        state = [x.clone() for x in (dev.k, dev.v, dev.k_scale, dev.v_scale)]
        dev.seq_len += 1


@gpu
def test_calls_on_a_given_stream_and_repeatable():
    """The stream argument, and the same bits on every run."""
    m = q()
    c = Pages([3000, 2500], [3000, 3000], 2, 128, 64, 13, scales=(-9, -5))
    dev = c.cuda()
    Q = randn(5, 2, 8, 1, 128).to(torch.bfloat16).cuda()
    torch.cuda.synchronize()
    want = None
    for k in range(4):
        s = torch.cuda.Stream() if k % 2 else None
        idx, cnt, _, _ = m.quoka_cache_select(Q, dev, 3000, 1, 300, stream=s)
        O, lse = m.quoka_cache_attn(Q, dev, 3000, idx, cnt, want_lse=True, stream=s)
        A, _ = m.quoka_cache_attn(Q, dev, 3000, stream=s)
        torch.cuda.synchronize()
        got = [x.clone() for x in (idx, cnt, O, lse, A)]
        want = want or got
        assert all(torch.equal(x, y) for x, y in zip(got, want))


class Fenced:
    """A buffer of n bytes between two runs of 4 KB that no call may touch."""

    def __init__(self, n):
        self.raw = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
        self.ws = self.raw[4096:4096 + n]

    def like(self, shape, dtype):
        return self.ws.view(dtype).view(shape)

    def whole(self):
        return bool((self.raw[:4096] == 0xA5).all() and (self.raw[4096 + self.ws.numel():] == 0xA5).all())


@gpu
@pytest.mark.parametrize("dt,BCP", [("bf16", 1), ("bf16", 70), ("f32", 40)])
def test_calls_write_only_inside_outputs_and_workspace(dt, BCP):
    """Outputs and workspaces of exactly the sizes asked for, fenced; keys and
    values are the two halves of one pool."""
    m, t, es = q(), TYPES[dt], torch.finfo(TYPES[dt]).bits // 8
    b, nkv, nq, d, page, held = 3, 2, 6, 64, 32, [50, 0, 131]
    c = Pages(held, [n + BCP for n in held], nkv, d, page, 21, scales=(-9, -5))
    pool = torch.stack((c.k, c.v), 1).cuda()  # (npages, 2, nkv, page, d)
    before = pool.clone()
    cache = m.QuokaCache(pool[:, 0], pool[:, 1], c.k_scale.cuda(), c.v_scale.cuda(), c.table.cuda(),
                         torch.tensor(held, dtype=torch.int32).cuda())
    K, V, Q = (randn(s, b, h, BCP, d).to(t).cuda() for s, h in ((1, nkv), (2, nkv), (3, nq)))
    cos, sin = (x.cuda() for x in angles(200 + BCP, 32))
    kr, qr, st = Fenced(K.numel() * es), Fenced(Q.numel() * es), Fenced(256)
    Kr, Qr = kr.like(K.shape, t), qr.like(Q.shape, t)
    m.quoka_cache_append(cache, K, V, Q, cos, sin, Kr=Kr, Qr=Qr, ws=st.ws)
    touched = torch.zeros(pool.shape[0], page, dtype=torch.bool)
    for i, n in enumerate(held):
        for pos in range(n // page * page, n + BCP):  # a half-full page may be brought to a new scale
            touched[int(c.table[i, pos // page]), pos % page] = True
    same = (pool == before).all(-1).all(2).all(1).cpu()
    assert same[~touched].all() and kr.whole() and qr.whole() and st.whole()
    cache.seq_len += BCP
    L, NQ, BSA = 131 + BCP, min(2, BCP), 40
    pool0, scales0 = pool.clone(), cache.k_scale.clone()
    n = m.quoka_select_workspace_size(b, nq, nkv, d, L, BCP, NQ, BSA, t)
    ws, ix, ct, sc = Fenced(n), Fenced(b * nkv * BSA * 4), Fenced(b * nkv * 4), Fenced(b * nkv * L * 4)
    idx, cnt = ix.like((b, nkv, BSA), torch.int32), ct.like((b, nkv), torch.int32)
    m.quoka_cache_select(Qr, cache, L, NQ, BSA, kv_idx=idx, kv_count=cnt, s_agg=sc.like((b, nkv, L), torch.float32), ws=ws.ws)
    assert ws.whole() and ix.whole() and ct.whole() and sc.whole() and m.quoka_get_device_status(ws.ws) == 0
    for args, N in (((idx, cnt), BSA), ((), L)):
        ks, vs = Fenced(b * nkv * N * d * es), Fenced(b * nkv * N * d * es)
        m.quoka_cache_gather(cache, L, *args, dtype=t, Ksel=ks.like((b, nkv, N, d), t), Vsel=vs.like((b, nkv, N, d), t), ws=st.ws)
        assert ks.whole() and vs.whole() and st.whole()
        for own in ((K, V), (None, None)):
            n = m.quoka_cache_attn_workspace_size(b, nq, nkv, d, BCP, N, t)
            ws, o, ls = Fenced(n), Fenced(Q.numel() * es), Fenced(b * nq * BCP * 4)
            O, lse = o.like(Q.shape, t), ls.like((b, nq, BCP), torch.float32)
            m.quoka_cache_attn(Qr, cache, L, *(args or (None, None)), *own, O=O, lse=lse, ws=ws.ws)
            assert ws.whole() and o.whole() and ls.whole() and m.quoka_get_device_status(ws.ws) == 0
            assert O.isfinite().all() and lse.isfinite().all()
    assert torch.equal(pool, pool0) and torch.equal(cache.k_scale, scales0)


@gpu
def test_two_streams_at_once():
    """Two calls on two streams with workspaces of their own give what they
    give one after the other."""
    m = q()
    jobs = []
    for k, (BCP, dt) in enumerate(((1, "bf16"), (90, "bf16"), (5, "f32"))):
        c = Pages([3000, 1000], [3000, 1000], 2, 128, 64, 30 + k, scales=(-9, -5)).cuda()
        jobs.append((randn(40 + k, 2, 8, BCP, 128).to(TYPES[dt]).cuda(), c))

    def work(Q, c, s=None):
        idx, cnt, _, _ = m.quoka_cache_select(Q, c, 3000, 1, 200, stream=s)
        return [m.quoka_cache_attn(Q, c, 3000, stream=s)[0], m.quoka_cache_attn(Q, c, 3000, idx, cnt, stream=s)[0], cnt]

    want = [work(*j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(5):
        got = [work(*j, s) for j, s in zip(jobs, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(g, w))


@gpu
def test_two_threads_at_once(lib):  # noqa: F811
    """The C entry points from two threads (ctypes lets go of the interpreter's
    lock), each on a stream of its own, with sizes that need different amounts of
    shared memory of the same kernels: no call is refused, and the results are
    those of one thread."""
    m = q()
    sizes = [(2900, 200, 8), (9000, 500, 24)]  # keys, chunk of the select, its NQ
    jobs = []
    for k, (n, BCP, NQ) in enumerate(sizes):
        c = Pages([n], [n], 2, 128, 64, 60 + k, scales=(-9, -5)).cuda()
        Qs, Qa = randn(61 + k, 1, 4, BCP, 128).to(torch.bfloat16).cuda(), randn(63 + k, 1, 4, 8 + 12 * k, 128).cuda()
        idx, cnt, _, _ = m.quoka_cache_select(Qs, c, n, NQ, 100)
        O, _ = m.quoka_cache_attn(Qa, c, n)
        jobs.append((c, n, NQ, Qs, Qa, idx, cnt, O))
    torch.cuda.synchronize()
    faults = []

    def work(k):
        try:
            c, n, NQ, Qs, Qa, idx, cnt, O = jobs[k]
            tv = m._lib.tensor_view
            stream = torch.cuda.Stream()
            idx1, cnt1, O1 = torch.zeros_like(idx), torch.zeros_like(cnt), torch.zeros_like(O)
            wn = lib.quoka_select_workspace_size(1, 4, 2, 128, n, Qs.shape[2], NQ, 100, 1)
            an = lib.quoka_cache_attn_workspace_size(1, 4, 2, 128, Qa.shape[2], n, 0)
            ws, wa = (torch.zeros(x, dtype=torch.uint8, device="cuda") for x in (wn, an))
            torch.cuda.synchronize()
            p, B, vs, va = (lambda t: ctypes.c_void_p(t.data_ptr())), ctypes.byref, tv(Qs), tv(Qa)
            for _ in range(300):
                r = lib.quoka_cache_select(B(vs), B(c._view), n, NQ, 100, p(idx1), p(cnt1), None, None, p(ws), wn,
                                           ctypes.c_void_p(stream.cuda_stream))
                r2 = lib.quoka_cache_attn(B(va), B(c._view), n, None, None, n, None, None, 128**-0.5, p(O1), None, p(wa), an,
                                          ctypes.c_void_p(stream.cuda_stream))
                if r or r2:
                    faults.append((k, r, r2))
                    break
            stream.synchronize()
            if not (torch.equal(idx, idx1) and torch.equal(cnt, cnt1) and torch.equal(O, O1)):
                faults.append((k, "results"))
        except BaseException as e:  # (a thread's failure is the test's)
            faults.append((k, repr(e)))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not faults


def given_up(kind, call, ws):
    """Runs call() with the waits bounded by 5 ms and the barrier of `kind` expecting
    an arrival that never comes; the status and fault site of ws."""
    q().quoka_debug_set_wait_hooks(5_000_000, kind)
    try:
        call()
        torch.cuda.synchronize()
    finally:
        q().quoka_debug_set_wait_hooks()
    return q().quoka_get_device_status(ws), q().quoka_get_device_fault_site(ws)


@gpu
@pytest.mark.parametrize("NQ,d", [(2, 64), (2, 128), (40, 64), (100, 128)])
def test_scoring_that_gives_up_unwinds(NQ, d):
    """A wait that runs out is QUOKA_ERR_TIMEOUT with its site and a count of 0 (no
    stale selection); the same call, workspace and device then give what they gave
    before. One sequence, long enough that every range has more tiles than stages."""
    m, n, BCP = q(), 200_000, 2 * NQ
    c = Pages([n], [n], 1, d, 128, 7).cuda()
    Q = randn(8, 1, 2, BCP, d).cuda()
    ws = torch.zeros(m.quoka_select_workspace_size(1, 2, 1, d, n, BCP, NQ, 900, Q.dtype), dtype=torch.uint8, device="cuda")
    idx, cnt = torch.zeros(1, 1, 900, dtype=torch.int32, device="cuda"), torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    s = torch.zeros(1, 1, n, device="cuda")
    call = lambda: m.quoka_cache_select(Q, c, n, NQ, 900, kv_idx=idx, kv_count=cnt, s_agg=s, ws=ws)
    call()
    want = idx.clone(), s.clone()
    for _ in range(3):
        status, site = given_up(m._lib.DEBUG_INJECT_CACHE_SCORE, call, ws)
        assert status == 5 and site in (63, 64, 65, 66) and int(cnt) == 0
        idx.fill_(-1)
        call()
        assert m.quoka_get_device_status(ws) == 0 and m.quoka_get_device_fault_site(ws) == 0
        assert int(cnt) == 900 and torch.equal(idx, want[0]) and torch.equal(s, want[1])


@gpu
@pytest.mark.parametrize("dt,d,BCP,listed", [("bf16", 128, 1, False), ("bf16", 64, 16, True), ("f32", 128, 1, True),
                                             ("f32", 64, 40, False)])
def test_attention_that_gives_up_unwinds(dt, d, BCP, listed):
    """The same of the attention over the codes, whose second kernel reports the
    first one's faults."""
    m, n = q(), 200_000
    c = Pages([n], [n], 1, d, 128, 7, scales=(-9, -5)).cuda()
    Q = randn(8, 1, 2, BCP, d).to(TYPES[dt]).cuda()
    idx = torch.randperm(n, generator=torch.Generator().manual_seed(1), dtype=torch.int32).view(1, 1, n).cuda() if listed else None
    cnt = torch.full((1, 1), n, dtype=torch.int32, device="cuda") if listed else None
    ws = torch.zeros(m.quoka_cache_attn_workspace_size(1, 2, 1, d, BCP, n, TYPES[dt]), dtype=torch.uint8, device="cuda")
    O = torch.zeros_like(Q)
    call = lambda: m.quoka_cache_attn(Q, c, n, idx, cnt, O=O, ws=ws)
    call()
    want = O.clone()
    for _ in range(3):
        status, site = given_up(m._lib.DEBUG_INJECT_CACHE_ATTN, call, ws)
        assert status == 5 and site in (61, 62)
        call()
        assert m.quoka_get_device_status(ws) == 0 and m.quoka_get_device_fault_site(ws) == 0 and torch.equal(O, want)


@gpu
@pytest.mark.parametrize("rows,T,BSA", [(20, 33000, 4000), (40, 20001, 100), (130, 9000, 8999), (600, 5000, 1), (74, 40000, 777)])
def test_topk_of_many_rows(rows, T, BSA):
    """Rows that alone fill the GPU take fewer, longer slices; values on a coarse
    grid, so that many are equal: ties go to the lower index."""
    s = (torch.randint(-200, 200, (rows, 1, T), generator=torch.Generator().manual_seed(rows)).float() / 200).cuda()
    idx, cnt = q().quoka_topk(s, BSA)
    want = s.sort(dim=-1, descending=True, stable=True).indices[..., :BSA].sort(-1).values
    assert (cnt == BSA).all() and torch.equal(idx.long(), want)


TIES = [
    # lens, kinds of keys (0: all different), how many keys in a row are of one kind, BSA
    ([3000, 2100, 0, 1], 0, 1, 700),
    ([8191, 5000, 900], 0, 1, 2048),
    ([8192, 4097], 150, 1, 3000),       # some fifty equal keys at the threshold
    ([8000], 7, 1, 1234),               # over a thousand
    ([32768], 0, 1, 4096),              # a cluster of CTAs
    ([30001], 120, 1, 4001),
    ([30000], 60, 500, 7777),           # equal keys lie together: in the slices of one or two CTAs
    ([32000, 17], 5, 1, 9999),
    ([20000], 1, 1, 19999),             # all equal
    ([50000], 0, 1, 1),
    ([70000], 300, 7, 12345),           # more than the registers hold
    ([9000] * 80, 400, 3, 500),
]


@gpu
@pytest.mark.parametrize("k", range(len(TIES)))
def test_select_takes_the_first_of_equal_scores(k):
    """Picks against a stable sort of the call's own scores."""
    lens, kinds, run, BSA = TIES[k]
    b, d, page, most = len(lens), 64, 128, max(lens)
    npp = (most + page - 1) // page
    g = torch.Generator().manual_seed(k)
    rows = torch.randint(0, 119, (kinds or b * npp * page, d), generator=g, dtype=torch.uint8)
    rows |= torch.randint(0, 2, rows.shape, generator=g, dtype=torch.uint8) << 7
    if kinds:
        rows = rows[torch.randint(0, kinds, ((b * npp * page + run - 1) // run,), generator=g).repeat_interleave(run)[:b * npp * page]]
    codes = rows.reshape(b * npp, 1, page, d).cuda()
    scale, table = torch.ones(b * npp, 1, device="cuda"), torch.arange(b * npp, dtype=torch.int32).reshape(b, npp).cuda()
    c = q().QuokaCache(codes, codes.clone(), scale, scale.clone(), table, torch.tensor(lens, dtype=torch.int32).cuda())
    Q = randn(k, b, 2, 5, d).cuda()
    idx, count, _, s = q().quoka_cache_select(Q, c, most, 2, BSA, want_s_agg=True)
    for i, n in enumerate(lens):
        m = min(n, BSA)
        assert int(count[i, 0]) == m
        want = s[i, 0, :n].sort(descending=True, stable=True).indices[:m].sort().values
        assert torch.equal(idx[i, 0, :m].long(), want)


@gpu
def test_no_room_for_an_output_or_a_workspace():
    """torch.OutOfMemoryError, as of the package's other calls, and the next call
    works: outputs of 2^40 bytes and more that no device has room for."""
    m, page, cols = q(), 128, 2**21
    table = torch.zeros(1, cols, dtype=torch.int32, device="cuda")
    k = torch.zeros(1, 8, page, 128, dtype=torch.uint8, device="cuda")
    c = m.QuokaCache(k, k.clone(), torch.ones(1, 8, device="cuda"), torch.ones(1, 8, device="cuda"), table,
                     torch.full((1,), 5, dtype=torch.int32, device="cuda"))
    Q = torch.ones(1, 8, 64, 128, device="cuda", dtype=torch.bfloat16)
    n = page * cols  # 2^28 rows
    with pytest.raises(torch.OutOfMemoryError):
        m.quoka_cache_gather(c, n, dtype=torch.float32)
    with pytest.raises(torch.OutOfMemoryError):
        m.quoka_cache_attn(Q, c, n)  # (the dequantised rows are its workspace)
    O, _ = m.quoka_cache_attn(Q, c, 5)
    assert torch.equal(O, torch.zeros_like(O))


@gpu
def test_long_table_offsets_pass_32_bits():
    """A pool of more than 2^32 bytes, with the pages of a sequence at both ends."""
    page, nkv, d = 128, 8, 128
    npages = (2**32 + 2**28) // (page * nkv * d)
    k = torch.zeros(npages, nkv, page, d, dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    scale = torch.ones(npages, nkv, device="cuda")
    table = torch.tensor([[npages - 1, 0, npages - 2]], dtype=torch.int32, device="cuda")
    seq = torch.zeros(1, dtype=torch.int32, device="cuda")
    c = q().QuokaCache(k, v, scale, scale.clone(), table, seq)
    K, V = (randn(s, 1, nkv, 300, d).to(torch.bfloat16).cuda() for s in (1, 2))
    q().quoka_cache_append(c, K, V)
    seq.fill_(300)
    Kg, Vg = q().quoka_cache_gather(c, 300)
    for x, y in ((Kg, K), (Vg, V)):  # e4m3: half a step is 2^-4; below 2^-6 of the scale, half of 2^-9 of it
        assert ((x.double() - y.double()).abs() <= 2.0**-4 * y.double().abs() + 2.0**-10 * 2.0**-5).all()
    Q = randn(3, 1, 8, 1, d).to(torch.bfloat16).cuda()
    O, _ = q().quoka_cache_attn(Q, c, 300)
    cnt = torch.full((1, nkv), 300, dtype=torch.int32, device="cuda")
    idx = torch.arange(300, dtype=torch.int32, device="cuda").expand(1, nkv, 300).contiguous()
    O2, _ = q().quoka_cache_attn(Q, c, 300, idx, cnt)
    assert torch.equal(O, O2) and O.abs().sum() > 0


# ------------------------------------------------------------ host side

def cpu_cache(**kw):
    a = dict(k=torch.zeros(5, 2, 16, 64, dtype=torch.uint8), v=torch.zeros(5, 2, 16, 64, dtype=torch.uint8),
             k_scale=torch.ones(5, 2), v_scale=torch.ones(5, 2), page_table=torch.zeros(3, 4, dtype=torch.int32),
             seq_len=torch.zeros(3, dtype=torch.int32))
    a.update(kw)
    return q().QuokaCache(**a)


def test_cache_refuses_bad_tensors():
    cpu_cache()
    cpu_cache(k=torch.zeros(5, 16, 2, 64, dtype=torch.uint8).transpose(1, 2),
              v=torch.zeros(5, 16, 2, 64, dtype=torch.uint8).transpose(1, 2))
    for kw in ({"k": torch.zeros(5, 2, 16, 96, dtype=torch.uint8), "v": torch.zeros(5, 2, 16, 96, dtype=torch.uint8)},
               {"k": torch.zeros(5, 2, 24, 64, dtype=torch.uint8), "v": torch.zeros(5, 2, 24, 64, dtype=torch.uint8)},
               {"v": torch.zeros(5, 2, 32, 64, dtype=torch.uint8)}, {"k_scale": torch.ones(5, 3)},
               {"v": torch.zeros(5, 16, 2, 64, dtype=torch.uint8).transpose(1, 2)},
               {"v_scale": torch.ones(2, 5).t()}, {"page_table": torch.zeros(4, dtype=torch.int32)},
               {"page_table": torch.zeros(4, 3, dtype=torch.int32).t()}, {"seq_len": torch.zeros(2, dtype=torch.int32)}):
        with pytest.raises(ValueError):
            cpu_cache(**kw)
    for kw in ({"v": torch.zeros(5, 2, 16, 64)}, {"k_scale": torch.ones(5, 2, dtype=torch.float64)},
               {"seq_len": torch.zeros(3, dtype=torch.int64)}):
        with pytest.raises(TypeError):
            cpu_cache(**kw)


def test_cache_refuses_a_page_table_of_overlapping_rows():
    """Rows of a table are table_stride >= max_pages entries apart: one row for all
    sequences would be read past its end."""
    row = torch.zeros(1, 4, dtype=torch.int32)
    assert cpu_cache(page_table=row, seq_len=torch.zeros(1, dtype=torch.int32))._view.table_stride == 4
    assert cpu_cache(page_table=torch.zeros(3, 9, dtype=torch.int32)[:, :4])._view.table_stride == 9
    for table in (row.expand(3, 4), torch.zeros(9, dtype=torch.int32).as_strided((3, 4), (2, 1))):
        with pytest.raises(ValueError):
            cpu_cache(page_table=table)


def test_calls_refuse_bad_tensors(lib):  # noqa: F811
    m, c = q(), cpu_cache()
    K, Q = torch.zeros(3, 2, 7, 64), torch.zeros(3, 4, 7, 64)
    i32 = torch.int32
    for call in (lambda: m.quoka_cache_append(c, K, K),  # a cache on the CPU
                 lambda: m.quoka_cache_append(c, K, K[:, :, :6]),
                 lambda: m.quoka_cache_append(c, K, K, torch.zeros(3, 4, 6, 64)),
                 lambda: m.quoka_cache_append(c, K, K, Qr=Q),
                 lambda: m.quoka_cache_append(c, K, K, Q, torch.zeros(9, 32)),
                 lambda: m.quoka_cache_append(c, K, K, Kr=torch.zeros(3, 2, 8, 64)),
                 lambda: m.quoka_cache_append(c, K, K, new_len=torch.zeros(2, dtype=i32)),
                 lambda: m.quoka_cache_select(torch.zeros(2, 4, 7, 64), c, 10, 1, 1),
                 lambda: m.quoka_cache_select(Q, c, 10, 1, 5, kv_idx=torch.zeros(3, 2, 6, dtype=i32)),
                 lambda: m.quoka_cache_gather(c, 10, torch.zeros(3, 2, 6, dtype=i32)),
                 lambda: m.quoka_cache_gather(c, 10, torch.zeros(3, 2, 6, dtype=i32), torch.zeros(3, 3, dtype=i32)),
                 lambda: m.quoka_cache_attn(torch.zeros(3, 4, 7, 128), c, 10),
                 lambda: m.quoka_cache_attn(Q, c, 10, Kc=K),
                 lambda: m.quoka_cache_attn(Q, c, 10, None, None, K, K, O=torch.zeros(3, 4, 7, 64).transpose(1, 2))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: m.quoka_cache_append(c, K, K, new_len=torch.zeros(3)),
                 lambda: m.quoka_cache_append(c, K, None),
                 lambda: m.quoka_cache_append(c, K, K, Q=3),
                 lambda: m.quoka_cache_select(Q, c, 10.5, 1, 1),
                 lambda: m.quoka_cache_attn(Q, c, 10, scale="x"),
                 lambda: m.quoka_cache_append(c, K.half(), K.half()),
                 lambda: m.quoka_cache_gather(c, 10, dtype=torch.float16),
                 lambda: m.quoka_cache_attn(Q, c, 10, lse=torch.zeros(3, 4, 7, dtype=torch.float64))):
        with pytest.raises(TypeError):
            call()


def test_padded_select_refuses_bad_counts(lib):  # noqa: F811
    m, c, Q = q(), cpu_cache(), torch.zeros(3, 4, 7, 64)
    for new in (torch.zeros(2, dtype=torch.int32), torch.zeros(3, 1, dtype=torch.int32), torch.zeros(6, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError, match="new_len"):
            m.quoka_cache_select(Q, c, 10, 1, 1, new_len=new)
    for new in (torch.zeros(3), [1, 2, 3]):
        with pytest.raises(TypeError, match="new_len"):
            m.quoka_cache_select(Q, c, 10, 1, 1, new_len=new)
    B, buf, ws = ctypes.byref, ctypes.c_void_p(0x200000), ctypes.c_void_p(0x100000)

    def select(new=buf, max_len=100, NQ=2, ws=ws, n=1 << 30, c=_cache()):
        return lib.quoka_cache_select_padded(B(_view((1, 4, 7, 128))), new, B(c), max_len, NQ, 10, buf, buf, None, None, ws, n, None)

    assert select(new=None) == 1 and select(max_len=129) == 1 and select(NQ=8) == 1 and select(NQ=0) == 1
    assert select(ws=None) == 3 and select(n=256) == 3 and select(c=_cache(page=24)) == 2 and select(c=_cache(k=None)) == 1


def _cache(**kw):
    from sparse_kv_selection_quoka_b200._lib import quoka_cache
    a = dict(k=0x10000, v=0x20000, k_scale=0x30000, v_scale=0x30100, npages=9, nkv=2, page=16, d=128,
             page_stride=2 * 16 * 128, head_stride=16 * 128, row_stride=128, page_table=0x40000, table_stride=8, b=1,
             max_pages=8, seq_len=0x50000)
    a.update(kw)
    return quoka_cache(**a)


def test_entry_points_reject_bad_arguments_on_host(lib):  # noqa: F811
    """Every refusal comes before anything is enqueued (no GPU here)."""
    B = ctypes.byref
    ws, buf, out = (ctypes.c_void_p(x) for x in (0x100000, 0x200000, 0x300000))
    Q, K = _view((1, 4, 7, 128)), _view((1, 2, 7, 128), data=0x60000)
    big = 1 << 30

    def select(c=_cache(), Q=Q, max_len=100, NQ=2, BSA=10, count=buf, ws=ws, n=big):
        return lib.quoka_cache_select(B(Q), B(c), max_len, NQ, BSA, buf, count, None, None, ws, n, None)

    def attn(c=_cache(), Q=Q, max_len=100, idx=None, count=None, N=100, Kc=K, Vc=K, scale=0.1, O=out, ws=ws, n=big):
        return lib.quoka_cache_attn(B(Q), B(c), max_len, idx, count, N, Kc and B(Kc), Vc and B(Vc), scale, O, None, ws, n,
                                    None)

    def gather(c=_cache(), max_len=100, idx=None, count=None, N=100, dtype=1, K=out, V=out, ws=None, n=0):
        return lib.quoka_cache_gather(B(c), max_len, idx, count, N, dtype, K, V, ws, n, None)

    def app(c=_cache(), K=K, V=K, Q=None, cos=None, sin=None, npos=0, rot=0, flags=0, Kr=None, Qr=None, ws=None, n=0):
        return lib.quoka_cache_append(B(c), K and B(K), V and B(V), Q and B(Q), cos, sin, npos, rot, flags, None, Kr, Qr, ws,
                                      n, None)

    for f in (select, attn, gather, app):
        for kw in (dict(k=None), dict(v=0x20008), dict(k_scale=None), dict(npages=0), dict(b=0), dict(max_pages=0),
                   dict(table_stride=7), dict(row_stride=64), dict(row_stride=136), dict(head_stride=-2048),
                   dict(page_stride=0), dict(seq_len=None), dict(page_table=None)):
            assert f(_cache(**kw)) == 1, kw
        assert f(_cache(page=24)) == 2 and f(_cache(d=96)) == 2
    for f in (select, attn, gather):
        assert f(max_len=-1) == 1 and f(max_len=129) == 1  # 8 pages of 16 tokens
    assert select(NQ=0) == 1 and select(NQ=8) == 1 and select(BSA=-1) == 1 and select(count=None) == 1
    assert select(Q=_view((1, 3, 7, 128))) == 1 and select(Q=_view((2, 4, 7, 128))) == 1
    assert select(ws=None) == 3 and select(n=256) == 3 and select(ws=ctypes.c_void_p(0x100010)) == 3
    assert attn(Kc=None) == 1 and attn(scale=0.0) == 1 and attn(scale=float("nan")) == 1 and attn(O=None) == 1
    assert attn(N=99) == 1 and attn(idx=buf) == 1 and attn(idx=buf, count=buf, N=-1) == 1
    assert attn(Kc=_view((1, 2, 8, 128))) == 1 and attn(Q=_view((1, 4, 7, 128), dtype=0)) == 1
    need = lib.quoka_cache_attn_workspace_size(1, 4, 2, 128, 7, 100, 1)
    assert need > 256 and attn(n=need - 1) == 3
    assert lib.quoka_cache_attn_workspace_size(1, 4, 3, 128, 7, 100, 1) == 0
    assert lib.quoka_cache_attn_workspace_size(1, 4, 2, 96, 7, 100, 1) == 0
    assert gather(N=99) == 1 and gather(dtype=2) == 1 and gather(K=None) == 1 and gather(count=buf) == 1
    assert gather(ws=ctypes.c_void_p(0x100010), n=256) == 3
    assert app(K=None) == 1 and app(V=_view((1, 2, 8, 128))) == 1 and app(Q=Q) == 1 and app(Qr=out) == 1 and app(flags=2) == 1
    assert app(rot=8, cos=buf, sin=buf, npos=9) == 1 and app(rot=144, cos=buf, sin=buf, npos=9) == 1
    assert app(rot=16, cos=buf, sin=None, npos=9) == 1 and app(rot=16, cos=buf, sin=buf, npos=0) == 1
    # outputs over inputs
    assert app(Kr=ctypes.c_void_p(0x60000)) == 1 and app(Kr=ctypes.c_void_p(0x60000 + 256)) == 1
    assert app(Q=Q, Qr=ctypes.c_void_p(0x10000)) == 1


def test_cache_of_far_strides_is_refused_on_host(lib):  # noqa: F811
    """Before anything is enqueued, by every call (a size of one has no stride)."""
    B, ws, buf = ctypes.byref, ctypes.c_void_p(0x100000), ctypes.c_void_p(0x200000)
    far = 1 << 40
    for kw in (dict(page_stride=far), dict(head_stride=far), dict(row_stride=far)):
        c = _cache(**kw)
        assert lib.quoka_cache_select(B(_view((1, 4, 7, 128))), B(c), 100, 2, 10, buf, buf, None, None, ws, 1 << 30, None) == 2
        assert lib.quoka_cache_attn(B(_view((1, 4, 7, 128))), B(c), 100, None, None, 100, None, None, 0.1, buf, None, ws, 1 << 30,
                                    None) == 2
        assert lib.quoka_cache_gather(B(c), 100, None, None, 100, 1, buf, buf, None, 0, None) == 2
    none = _view((1, 1, 0, 128), data=None)
    one = _cache(npages=1, nkv=1, page_stride=far, head_stride=far)
    assert lib.quoka_cache_append(B(one), B(none), B(none), None, None, None, 0, 0, 0, None, None, None, None, 0, None) == 0


def test_append_of_an_empty_chunk_on_host(lib):  # noqa: F811
    """Nothing to do, whatever goes with it (an empty tensor's address is null)."""
    B, none = ctypes.byref, _view((1, 2, 0, 128), data=None)

    def app(Q=None, Qr=None):
        return lib.quoka_cache_append(B(_cache()), B(none), B(none), Q and B(Q), None, None, 0, 0, 0, None, None, Qr, None, 0,
                                      None)

    assert app() == 0 and app(Q=_view((1, 4, 0, 128), data=None)) == 0
    assert app(Q=_view((1, 4, 1, 128))) == 1 and app(Qr=ctypes.c_void_p(0x300000)) == 1


def test_tensor_map_encoder_is_found_by_every_thread(tmp_path):
    """First calls from many threads at once, while the driver takes its time to
    name the encoder: every one of them gets it (a fake of the runtime's lookup;
    no GPU). A lookup that fails is made again."""
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.NVCC)), "include")
    src = tmp_path / "first.cpp"
    src.write_text(r"""
#include <atomic>
#include "tmap.cuh"
#include <chrono>
#include <cstdio>
#include <thread>
#include <vector>
static std::atomic<int> lookups{0}, fail{1};
static CUresult encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                       const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                       CUtensorMapL2promotion, CUtensorMapFloatOOBfill) { return CUDA_SUCCESS; }
extern "C" cudaError_t cudaGetDriverEntryPoint(const char*, void** p, unsigned long long,
                                               cudaDriverEntryPointQueryResult* q) {
  ++lookups;
  std::this_thread::sleep_for(std::chrono::milliseconds(100));
  if (fail) return cudaErrorUnknown;
  *p = (void*)&encode;
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
int main() {
  if (quoka::tensor_map_encoder() != nullptr) return 1;
  fail = 0;
  std::atomic<int> ready{0}, missed{0};
  std::vector<std::thread> ts;
  for (int i = 0; i < 8; ++i)
    ts.emplace_back([&] {
      ++ready;
      while (ready < 8) std::this_thread::yield();
      CUtensorMap m;
      if (!quoka::encode_codes_4d(&m, nullptr, 128, 64, 2, 3, 128, 8192, 16384, 64)) ++missed;
    });
  for (auto& t : ts) t.join();
  const int n = lookups;
  quoka::tensor_map_encoder();
  printf("%d %d\n", (int)missed, (int)lookups - n);
  return 0;
}
""")
    exe = tmp_path / "first"
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-I", build.CSRC, "-isystem", cuda, str(src), "-o", str(exe),
                    "-pthread"], check=True, capture_output=True, text=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=60).stdout
    assert out.split() == ["0", "0"], "threads without the encoder; lookups once it is known"


FIRST_CALLS = r"""
import sys, threading, torch
sys.path.insert(0, sys.argv[1])
import sparse_kv_selection_quoka_b200 as q
c = [q.QuokaCache(*(torch.zeros(9, 2, 16, 128, dtype=torch.uint8, device="cuda") + 56 for _ in "kv"),
                  *(torch.ones(9, 2, device="cuda") for _ in "kv"), torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8),
                  torch.full((1,), 120, dtype=torch.int32, device="cuda")) for _ in range(4)]
Q = torch.ones(1, 4, 1, 128, device="cuda", dtype=torch.bfloat16)
torch.cuda.synchronize()
gate, out = threading.Barrier(4), [None] * 4
def work(k):
    gate.wait()
    try:
        s = torch.cuda.Stream()
        idx, n, _, _ = q.quoka_cache_select(Q, c[k], 120, 1, 10, stream=s)
        O, _ = q.quoka_cache_attn(Q, c[k], 120, stream=s)
        s.synchronize()
        out[k] = (idx.tolist(), n.tolist(), O.float().sum().item())
    except Exception as e:
        out[k] = repr(e)
ts = [threading.Thread(target=work, args=(k,)) for k in range(4)]
[t.start() for t in ts]
[t.join() for t in ts]
assert all(o == ([[list(range(10))] * 2], [[10, 10]], 512.0) for o in out), out
print("same")
"""


@gpu
def test_first_calls_of_a_process_from_several_threads():
    """The package's calls as the first of a process, from four threads at once."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS, root], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]
