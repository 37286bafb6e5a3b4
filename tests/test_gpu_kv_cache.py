"""GPU checks of the key/value cache operators against 64-bit references: rotary
positions, appending and reading records, attention of drafted tokens, commit.

Bars (u(t) = finfo(t).eps / 2, the largest relative rounding of type t):
  * records without rotation: codes and scales bit for bit the oracle's;
  * records with rotation: a code may differ from the 64-bit value's only where
    that value lies within 1e-5 of a threshold, a scale by one fp16 step;
  * read: fp32 butterflies of 32 terms, five additions deep, three products:
    8 u(fp32) of the block's largest possible sum, plus the output's rounding;
  * rope: angle to 2^-25 turns (1.9e-7 rad) and the two fp32 functions to 2
    units, two products and a sum: 6e-7 (|x| + |y|), plus the output's rounding;
  * attention: three roundings to fp16 enter a score (query, centroid, centroid
    times scale), three a weighted value (weight, centroid, centroid times
    scale).  Each is at most 2^-11 relative and has an rms of 2^-11 / sqrt(3),
    independent from element to element, so a score is off by 2^-11 |q' . k'|
    rms (element products, 2-norm, times the softmax scale) and a row by
    2^-11 (1 + s) sqrt(sum p_j^2 |v_j|^2) rms with s the largest of these: the
    bar is four times that in 2-norm, plus the output's rounding.
"""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
CENTROIDS = [0.128395036, 0.388048291, 0.656759143, 0.942340434, 1.25623119, 1.6180464, 2.06901717, 2.73258948]
THRESHOLDS = [0.258221656, 0.522403717, 0.799549758, 1.09928584, 1.4371388, 1.84353185, 2.40080333]


def u(dtype):
    return torch.finfo(dtype).eps / 2


def _rand(seed, *shape, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def _hadamard():
    h = torch.ones(1, 1, dtype=torch.float64)
    for _ in range(5):
        h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)))
    return h


def _signs(dim):
    s = []
    for k in range(dim):
        h = k * 0x9E3779B9 % 2 ** 32
        h = (h ^ h >> 16) * 0x85EBCA6B % 2 ** 32
        s.append(-1.0 if (h ^ h >> 13) >= 2 ** 31 else 1.0)
    return torch.tensor(s, dtype=torch.float64)


def _rotated_domain(codes, scales):
    """Records (..., D/2), (..., D/16) to c * d, fp64."""
    table = torch.tensor(CENTROIDS + [-c for c in CENTROIDS]).double()
    c = torch.stack((table[(codes & 15).long()], table[(codes >> 4).long()]), -1).flatten(-2)
    return c * scales.view(F16).double().repeat_interleave(16, -1)


def _back(y):
    """s . (H y) / 32 per block."""
    D = y.shape[-1]
    return (y.reshape(-1, 32) @ _hadamard()).reshape(y.shape) * _signs(D) / 32


def _forward(x):
    return ((x.double() * _signs(x.shape[-1])).reshape(-1, 32) @ _hadamard()).reshape(x.shape)


def _values(codes, scales):
    return _back(_rotated_domain(codes.cpu(), scales.cpu()))


def _rope_ref(x, positions, inv_freq, interleaved, scale=1.0, inverse=False):
    out = x.double().clone()
    a = positions.double()[:, None] * inv_freq.double()
    if inverse:
        a = -a
    c, s = (a.cos() * scale)[:, None], (a.sin() * scale)[:, None]
    h = inv_freq.numel()
    i, j = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
    p, q = x[..., i].double(), x[..., j].double()
    out[..., i], out[..., j] = p * c - q * s, p * s + q * c
    size = x.double().abs()
    size[..., i] = size[..., j] = x[..., i].double().abs() + x[..., j].double().abs()
    return out, size * max(1.0, abs(scale))


def _i32(v):
    return torch.as_tensor(v, dtype=torch.int32).to(DEV)


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n,heads,dim,rot,interleaved", [
    (1, 1, 2, 2, False), (1, 32, 128, 128, False), (7, 3, 64, 64, True), (33, 5, 96, 32, True),
    (129, 2, 128, 90, False), (5, 7, 50, 34, True), (257, 8, 256, 128, False), (3, 1, 1024, 1022, True),
    (4000, 16, 128, 64, False)])
def test_rope(cuda_lib, dtype, n, heads, dim, rot, interleaved):
    x = _rand(n * dim, n, heads, dim, dtype=dtype)
    g = torch.Generator().manual_seed(n)
    pos = torch.randint(-1000, 2 ** 31 - 1, (n,), generator=g).to(torch.int32)
    pos[: n // 2] %= 5000
    f = cuda_lib.rope_frequencies(rot, 10000.0, device="cpu")
    got = cuda_lib.rope(x.to(DEV), pos.to(DEV), f.to(DEV), interleaved=interleaved, scale=1.25)
    ref, size = _rope_ref(x, pos, f, interleaved, 1.25)
    err = (got.cpu().double() - ref).abs()
    assert torch.all(err <= 6e-7 * size + u(dtype) * (ref.abs() + 6e-7 * size))
    if rot < dim:
        assert torch.equal(got.cpu()[..., rot:], x[..., rot:])


def test_rope_strides_in_place_and_back(cuda_lib):
    fused = _rand(1, 40, 3, 6, 128).to(DEV)  # q, k, v of a fused projection
    keep = fused.clone()
    pos, f = _i32(range(100, 140)), cuda_lib.rope_frequencies(96, 500000.0)
    q = fused[:, 1]
    want = cuda_lib.rope(q, pos, f)
    assert cuda_lib.rope(q, pos, f, out=q) is q
    assert torch.equal(q, want)
    assert torch.equal(fused[:, 0], keep[:, 0]) and torch.equal(fused[:, 2], keep[:, 2])
    # odd strides and offsets run element by element
    odd = torch.zeros(40, 6, 131, device=DEV)[..., 3:]
    odd.copy_(keep[:, 1])
    assert torch.equal(cuda_lib.rope(odd, pos, f), want)
    # the inverse is the transpose: <rope x, y> = <x, rope^-1 y>, and at scale 1 it undoes the rotation
    y = _rand(2, 40, 6, 128).to(DEV)
    x = keep[:, 1].contiguous()
    a = (want.double() * y.double()).sum()
    b = (x.double() * cuda_lib.rope(y, pos, f, inverse=True).double()).sum()
    assert abs(a - b) <= 2e-6 * (x.double().abs() * y.double().abs()).sum() * 2
    again = cuda_lib.rope(want, pos, f, inverse=True)
    assert torch.all((again - x).abs() <= 4e-6 * x.abs().amax())
    assert cuda_lib.rope(x[:0], pos[:0], f).shape == (0, 6, 128)


def test_rope_gradient_by_differences(cuda_lib):
    n, D = 3, 16
    f, pos = cuda_lib.rope_frequencies(12), _i32([5, 900, 31])
    x, w = _rand(3, n, 2, D).to(DEV), _rand(4, n, 2, D).to(DEV)
    grad = cuda_lib.rope(w, pos, f, scale=0.5, inverse=True)
    h = 0.25  # linear, so differences of any step are exact up to rounding
    for e in range(D):
        step = torch.zeros_like(x)
        step[..., e] = h
        up, down = cuda_lib.rope(x + step, pos, f, scale=0.5), cuda_lib.rope(x - step, pos, f, scale=0.5)
        d = ((up - down).double() * w.double()).sum(-1) / (2 * h)
        assert torch.all((d - grad[..., e]).abs() <= 1e-5 * w.abs().amax() * 4)


# ---------------------------------------------------------------------------
# append and read
# ---------------------------------------------------------------------------
def _pool(tq, seqs, per_seq, kv_heads, dim, page, seed=0):
    """A cache whose sequences hold their pages in a mixed order."""
    codes, scales = tq.kv_cache(seqs * per_seq + 1, kv_heads, dim, page)
    order = torch.randperm(seqs * per_seq + 1, generator=torch.Generator().manual_seed(seed))[: seqs * per_seq]
    return codes, scales, order.to(torch.int32).view(seqs, per_seq).contiguous().to(DEV)


def _records(t, table, seqs, places):
    """t[page of (seq, place), :, :, row] of all tokens: [n, 2, kv_heads, ...], on the CPU."""
    page = t.shape[3]
    table, t = table.cpu().long(), t.cpu()
    s, p = torch.as_tensor(seqs).long(), torch.as_tensor(places).long()
    return t[table[s, p // page], :, :, p % page]


def _oracle_records(x):
    """The oracle's codes and scales of rows x [n, D], as cache records."""
    n, D = x.shape
    codes, scales = oracle.quantize(x.float().numpy())
    nsb = (D // 32 + 3) // 4
    codes = codes.reshape(-1, nsb, 16, 64).transpose(0, 2, 1, 3).reshape(-1, nsb, 64)[:n]
    j, L = np.arange(D // 2) // 16, np.arange(D // 2) % 16  # byte L of block j of the row
    c = codes[:, j // 4, 16 * (L % 4) + 4 * (j % 4) + L // 4]
    scales = scales.reshape(-1, nsb, 16, 8).transpose(0, 2, 1, 3).reshape(-1, nsb * 8)[:n, : D // 16]
    return torch.from_numpy(c.copy()), torch.from_numpy(scales.astype(np.uint16).view(np.int16).copy())


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n,seqs,kv,dim,page", [(1, 1, 1, 32, 16), (5, 2, 3, 64, 16), (37, 4, 2, 96, 32),
                                                (300, 3, 8, 128, 64), (64, 64, 8, 128, 16), (3, 2, 1, 256, 1024),
                                                (2000, 5, 5, 160, 128)])
def test_append_is_the_codec_and_read_undoes_it(cuda_lib, dtype, n, seqs, kv, dim, page):
    per = -(-(-(-n // seqs) + 5) // page)
    codes, scales, table = _pool(cuda_lib, seqs, per, kv, dim, page)
    s, p = [i % seqs for i in range(n)], [i // seqs + 5 for i in range(n)]
    x = _rand(n + dim, n, 2, kv, dim, dtype=dtype, scale=3.0)
    x[0, 0, 0] = 0  # a record of zeros
    fused = x.to(DEV)
    cuda_lib.kv_append(codes, scales, table, _i32(s), _i32(p), fused[:, 0], fused[:, 1])
    c, d = _records(codes, table, s, p), _records(scales, table, s, p)
    want_c, want_d = _oracle_records(x.reshape(-1, dim))
    assert torch.equal(c.reshape(-1, dim // 2), want_c)
    assert torch.equal(d.reshape(-1, dim // 16), want_d)
    # nothing else was written
    used = torch.zeros(codes.shape[0], page, dtype=torch.bool)
    used[table.cpu().long()[s, [q // page for q in p]], [q % page for q in p]] = True
    assert not codes.cpu().permute(0, 3, 1, 2, 4)[~used].any()
    assert not scales.cpu().permute(0, 3, 1, 2, 4)[~used].any()
    y = _rotated_domain(c, d)
    ref = _back(y)
    bound = (y.abs().reshape(-1, 32).sum(1, keepdim=True) / 32).expand(-1, 32).reshape(y.shape)
    for out in (F32, BF16, F16):
        k, v = cuda_lib.kv_read(codes, scales, table, _i32(s), _i32(p), dtype=out)
        got = torch.stack((k, v), 1).cpu().double()
        assert k.dtype == out
        # subnormal fp16 results round to the smallest step instead
        tol = 8 * u(F32) * bound + u(out) * (ref.abs() + 8 * u(F32) * bound) + torch.finfo(out).smallest_normal * torch.finfo(out).eps
        assert torch.all((got - ref).abs() <= tol)


# (n = 150: eight lanes a block; more: a block per lane, or eight lanes where the halves are no whole blocks)
@pytest.mark.parametrize("rot,interleaved,dtype,dim,n", [(128, False, F32, 128, 150), (128, True, BF16, 128, 150),
                                                         (64, False, F16, 96, 150), (50, False, F32, 64, 150),
                                                         (6, True, BF16, 32, 150), (256, False, BF16, 256, 150),
                                                         (128, False, BF16, 128, 3001), (96, True, F16, 128, 2999),
                                                         (64, False, F32, 96, 4001), (96, False, BF16, 128, 3001),
                                                         (256, False, F32, 256, 1500)])
def test_append_rotates_keys(cuda_lib, rot, interleaved, dtype, dim, n):
    kv, page = 3, 32
    codes, scales, table = _pool(cuda_lib, 2, -(-n // 2 // page) + 1, kv, dim, page)
    s, p = [i % 2 for i in range(n)], [i // 2 for i in range(n)]
    k, v = _rand(1, n, kv, dim, dtype=dtype), _rand(2, n, kv, dim, dtype=dtype)
    pos = torch.randint(0, 2000000, (n,), generator=torch.Generator().manual_seed(3)).to(torch.int32)
    f = cuda_lib.rope_frequencies(rot, 500000.0, device="cpu")
    cuda_lib.kv_append(codes, scales, table, _i32(s), _i32(p), k.to(DEV), v.to(DEV),
                       rope=(pos.to(DEV), f.to(DEV)), interleaved=interleaved, rope_scale=1.1)
    c, d = _records(codes, table, s, p), _records(scales, table, s, p)
    want_c, want_d = _oracle_records(v.reshape(-1, dim))
    assert torch.equal(c[:, 1].reshape(-1, dim // 2), want_c) and torch.equal(d[:, 1].reshape(-1, dim // 16), want_d)
    y = _forward(_rope_ref(k, pos, f, interleaved, 1.1)[0])
    exact = y.reshape(n, kv, -1, 16).square().mean(-1).sqrt()
    assert torch.all((d[:, 0].to(torch.int32) - exact.half().view(torch.int16).to(torch.int32)).abs() <= 1)
    df = d[:, 0].view(F16).double()
    a = (y.abs().reshape(n, kv, -1, 16) / df[..., None]).reshape(n, kv, dim)
    rank = sum((a > t).to(torch.int64) for t in THRESHOLDS)
    got = torch.stack((c[:, 0] & 15, c[:, 0] >> 4), -1).flatten(-2).long()
    off = (got & 7) != rank
    near = torch.stack([(a - t).abs() for t in THRESHOLDS]).amin(0)
    assert torch.all(near[off] < 1e-5)
    sign_off = (got >> 3) != (y < 0)
    assert torch.all(a[sign_off] < 1e-5)


def test_append_drops_what_has_no_place(cuda_lib):
    codes, scales, table = _pool(cuda_lib, 2, 2, 2, 64, 16)
    codes.fill_(7)
    scales.fill_(9)
    table[1, 1] = 100  # outside the pool
    table[0, 1] = -1
    s = [-1, 2, 0, 0, 0, 1, 1, 2 ** 31 - 1, 0]
    p = [0, 0, -1, 32, 16, 16, 31, 0, 2 ** 31 - 1]
    x = _rand(5, len(s), 2, 64).to(DEV)
    cuda_lib.kv_append(codes, scales, table, _i32(s), _i32(p), x, x)
    assert torch.all(codes == 7) and torch.all(scales == 9)
    k, v = cuda_lib.kv_read(codes, scales, table, _i32(s), _i32(p))
    assert not k.any() and not v.any()
    none = _i32([])
    cuda_lib.kv_append(codes, scales, table, none, none, x[:0], x[:0])
    assert cuda_lib.kv_read(codes, scales, table, none, none)[0].shape == (0, 2, 64)


def test_append_saturates_and_stays_finite(cuda_lib):
    codes, scales, table = _pool(cuda_lib, 1, 1, 1, 64, 16)
    x = torch.zeros(4, 1, 64)
    x[0] = 60000.0
    x[1, 0, 3] = float("inf")
    x[2, 0, 40] = float("nan")
    x[3] = 1.0
    cuda_lib.kv_append(codes, scales, table, _i32([0] * 4), _i32(range(4)), x.to(DEV), x.to(DEV))
    d = _records(scales, table, [0] * 4, list(range(4))).view(F16).float()
    assert torch.all(d <= 23968.0) and torch.all(d >= 0)
    assert torch.all(torch.isfinite(cuda_lib.kv_read(codes, scales, table, _i32([0] * 4), _i32(range(4)), F32)[0]))
    # other blocks of the same record are untouched by the NaN
    assert torch.all(d[2, 0, 0, :2] == 0)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def _ancestors(parents, T):
    """Per token: the set it sees, or None if it is not there."""
    sees = []
    for i in range(T):
        par = i - 1 if parents is None else int(parents[i])
        if par < -1 or par >= i or (par >= 0 and sees[par] is None):
            sees.append(None)
        else:
            sees.append({i} | (sees[par] if par >= 0 else set()))
    return sees


def _attention_ref(codes, scales, table, lens, q, parents, scale, out_dtype):
    """(reference, bar in 2-norm per row), fp64."""
    B, T, H, D = q.shape
    kv, page = codes.shape[2], codes.shape[3]
    G = H // kv
    table, codes, scales = table.cpu().long(), codes.cpu(), scales.cpu()
    ref = torch.zeros(B, T, H, D, dtype=torch.float64)
    bar = torch.zeros(B, T, H, dtype=torch.float64)
    qr = _forward(q) / 32
    cap = table.shape[1] * page
    for b in range(B):
        n0 = min(max(int(lens[b]), 0), cap)
        n = min(n0 + T, cap)
        place = torch.arange(n)
        pages = table[b, place // page]
        good = (pages >= 0) & (pages < codes.shape[0])
        sees = _ancestors(None if parents is None else parents[b].tolist(), T)
        for h in range(kv):
            rows = pages.clamp(0, codes.shape[0] - 1), h, place % page
            k, v = (_rotated_domain(codes[rows[0], w, h, rows[2]], scales[rows[0], w, h, rows[2]]) for w in (0, 1))
            for t in range(T):
                if sees[t] is None:
                    continue
                ok = good & (place < n0)
                for j in sees[t]:
                    if n0 + j < n:
                        ok[n0 + j] = good[n0 + j]
                if not ok.any():
                    continue
                kk, vv = k[ok], v[ok]
                for g in range(G):
                    x = qr[b, t, h * G + g]
                    p = torch.softmax(kk @ x * scale, 0)
                    o = _back((p @ vv)[None])[0]
                    s = ((kk * x).norm(dim=1).amax() * abs(scale)).item()
                    spread = (p.square() * vv.square().sum(1) / 32).sum().sqrt().item()
                    ref[b, t, h * G + g] = o
                    bar[b, t, h * G + g] = 4 * 2.0 ** -11 * (1 + s) * spread + u(out_dtype) * o.norm().item()
    return ref, bar


def _filled(tq, B, per, kv, dim, page, seed):
    """A pool with every record written from Gaussian data."""
    codes, scales, table = _pool(tq, B, per, kv, dim, page, seed)
    n = per * page
    s = torch.arange(B).repeat_interleave(n)
    p = torch.arange(n).repeat(B)
    k, v = _rand(seed, B * n, kv, dim).to(DEV), _rand(seed + 1, B * n, kv, dim).to(DEV)
    tq.kv_append(codes, scales, table, _i32(s), _i32(p), k, v)
    return codes, scales, table


def _tree(seed, B, T, absent=False):
    g = torch.Generator().manual_seed(seed)
    par = torch.stack([torch.randint(-1, i, (B,), generator=g) if i else torch.full((B,), -1) for i in range(T)], 1)
    if absent:
        gone = torch.rand(B, T, generator=g) < 0.25
        par = torch.where(gone, torch.tensor([-2, 99, T, -100])[torch.randint(0, 4, (B, T), generator=g)], par)
    return par.to(torch.int32)


def _poison(codes, scales, table, lens, parents, T):
    """NaN scales wherever no row attends: behind the drafted tokens, and at absent ones."""
    page = codes.shape[3]
    cap = table.shape[1] * page
    bits = torch.tensor(float("nan")).half().view(torch.int16)
    for b in range(table.shape[0]):
        n0 = min(max(int(lens[b]), 0), cap)
        sees = _ancestors(None if parents is None else parents[b].tolist(), T)
        bad = [n0 + i for i in range(T) if sees[i] is None] + list(range(n0 + T, cap))
        bad = [i for i in bad if i < cap]
        if bad:
            at = table.cpu().long()[b, torch.tensor(bad) // page]
            scales[at.to(DEV), :, :, torch.tensor(bad).to(DEV) % page] = int(bits)
            codes[at.to(DEV), :, :, torch.tensor(bad).to(DEV) % page] = 255


CASES = [
    # B, T, heads, kv, dim, page, lens, dtype, tree
    (1, 1, 1, 1, 32, 16, [0], F16, None),
    (1, 1, 4, 1, 128, 16, [1], BF16, None),
    (2, 1, 8, 2, 64, 16, [15, 16], F32, None),
    (3, 1, 32, 8, 128, 64, [100, 0, 1023], BF16, None),
    (2, 1, 3, 3, 96, 32, [255, 17], F16, None),
    (2, 1, 8, 1, 256, 64, [300, 5], BF16, None),
    (2, 3, 6, 2, 160, 16, [77, 130], F16, "tree"),
    (1, 2, 16, 2, 128, 16, [2000], BF16, None),
    (3, 5, 6, 2, 64, 16, [31, 400, 0], F16, "tree"),
    (2, 16, 8, 2, 128, 64, [63, 500], BF16, "tree"),
    (2, 16, 8, 2, 128, 64, [640, 0], F32, "absent"),
    (2, 64, 8, 2, 128, 64, [64, 333], BF16, "tree"),
    (1, 64, 4, 4, 64, 32, [190], F16, "absent"),
    (2, 33, 3, 1, 96, 16, [129, 1], BF16, "tree"),
    (1, 64, 16, 1, 128, 128, [700], F16, None),
    (1, 7, 71, 1, 128, 16, [333], F16, "tree"),
    (1, 9, 8, 1, 256, 16, [222], BF16, "absent"),
    (40, 1, 4, 2, 64, 16, [7 * i for i in range(40)], F16, None),
    (1, 3, 2, 1, 192, 1024, [1500], BF16, "tree"),
    (2, 1, 16, 2, 224, 256, [0, 700], F16, None),
    (1, 5, 34, 2, 128, 512, [900], F32, "tree"),  # 85 rows on the tensor cores, some of a warp's missing
    (3, 50, 3, 1, 64, 16, [0, 128, 700], BF16, "absent"),  # 150 rows: a row tile of its own for the last 22
    (1, 1, 4, 1, 64, 1024, [45000], F16, None),  # more parts than a warp joins at once
    (1, 24, 4, 2, 128, 64, [30000], BF16, "tree"),
    # more sequences than a CTA has threads, for both kernels
    (1200, 1, 2, 1, 32, 16, [i % 15 for i in range(1200)], F16, None),
    (520, 17, 1, 1, 64, 16, [i % 31 for i in range(520)], BF16, None),
    # many rows, one long sequence among short ones: its rows are joined by more than a warp
    (40, 2, 16, 1, 32, 16, [3 * (i % 5) for i in range(39)] + [3000], BF16, "tree"),
    (20, 8, 16, 2, 64, 16, [10000] + [i % 7 for i in range(19)], F16, "absent"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "b%d_t%d_h%d_kv%d_d%d_p%d_%s" % (*c[:6], c[8] or "chain"))
def test_attention(cuda_lib, case):
    B, T, H, kv, D, page, lens, dtype, kind = case
    per = -(-(max(lens) + T) // page)
    codes, scales, table = _filled(cuda_lib, B, per, kv, D, page, seed=B * T + D)
    parents = None if kind is None else _tree(T + D, B, T, kind == "absent")
    _poison(codes, scales, table, lens, parents, T)
    q = _rand(H + T, B, T, H, D, dtype=dtype, scale=1.5)
    scale = D ** -0.5
    ref, bar = _attention_ref(codes, scales, table, lens, q, parents, scale, dtype)
    par = None if parents is None else parents.to(DEV)
    got = cuda_lib.kv_attention(codes, scales, table, _i32(lens), q.to(DEV), parents=par)
    assert got.dtype == dtype
    err = (got.cpu().double() - ref).norm(dim=-1)
    assert torch.all(err <= bar), (err / bar.clamp(min=1e-30)).amax()
    # run again: the same bits, whatever the workspace held
    ws = cuda_lib.kv_attention_workspace(B, T, H, kv, D).fill_(255)
    assert torch.equal(cuda_lib.kv_attention(codes, scales, table, _i32(lens), q.to(DEV), parents=par, ws=ws), got)
    assert cuda_lib.workspace_status(ws) == 0


@pytest.mark.parametrize("out_dtype", [F32, BF16, F16])
def test_attention_strides_and_output_types(cuda_lib, out_dtype):
    B, T, H, kv, D, page = 2, 4, 8, 2, 128, 16
    lens = [50, 90]
    codes, scales, table = _filled(cuda_lib, B, 6, kv, D, page, seed=9)
    wide = _rand(1, T, B, H + 3, D + 32, dtype=BF16).to(DEV)
    q = wide.permute(1, 0, 2, 3)[:, :, 2:2 + H, :D]
    big = torch.full((B, T, H + 2, D + 16), 5.0, dtype=out_dtype, device=DEV)
    out = big[:, :, 1:1 + H, 8:8 + D]
    ref, bar = _attention_ref(codes, scales, table, lens, q.cpu(), None, 0.2, out_dtype)
    cuda_lib.kv_attention(codes, scales, table, _i32(lens), q, scale=0.2, out=out)
    assert torch.all((out.cpu().double() - ref).norm(dim=-1) <= bar)
    out.fill_(5.0)
    assert torch.all(big == 5.0)  # nothing beside the output was written


def test_attention_scores_of_any_size(cuda_lib):
    """Scores far apart (one weight near 1, the others underflowing), scale 0 and a negative scale."""
    B, T, H, kv, D, page = 1, 1, 4, 1, 128, 16
    codes, scales, table = _filled(cuda_lib, B, 20, kv, D, page, seed=21)
    lens = [300]
    for size, scale in ((40.0, 1.0), (1.0, 0.0), (2.0, -0.3), (300.0, 1.0)):
        q = _rand(5, B, T, H, D, dtype=BF16, scale=size)
        got = cuda_lib.kv_attention(codes, scales, table, _i32(lens), q.to(DEV), scale=scale, dtype=F32)
        assert torch.all(torch.isfinite(got))
        if size < 10:  # beyond that a score's rounding alone decides between near ties
            ref, bar = _attention_ref(codes, scales, table, lens, q, None, scale, F32)
            assert torch.all((got.cpu().double() - ref).norm(dim=-1) <= bar)
        else:  # the largest score's value, where the runner-up is far behind
            ref, _ = _attention_ref(codes, scales, table, lens, q, None, scale, F32)
            k = _rotated_domain(*(t[table.cpu().long()[0], 0, 0].reshape(-1, w)[:301] for t, w in
                                  ((codes.cpu(), D // 2), (scales.cpu(), D // 16))))
            z = (_forward(q)[0, 0] / 32) @ k.T * scale
            top = z.topk(2, dim=1).values
            clear = (top[:, 0] - top[:, 1]) > 60
            rel = (got.cpu().double() - ref)[0, 0].norm(dim=-1) / ref[0, 0].norm(dim=-1)
            assert torch.all(rel[clear] <= 3 * 2.0 ** -11)


def test_attention_small_weights_count(cuda_lib):
    """One token far above 8000 equal ones that together weigh as much: a weight of 2^-13 is not lost."""
    D, page, n = 64, 64, 8192
    codes, scales, table = cuda_lib.kv_cache(130, 1, D, page) + (_i32(range(130)).view(1, 130),)
    k = torch.zeros(n + 1, 1, D)
    k[n, 0, :] = 1.0  # the drafted token
    v = torch.ones(n + 1, 1, D)
    v[n] = -1.0
    zero = torch.zeros(n + 1, dtype=torch.int32, device=DEV)
    cuda_lib.kv_append(codes, scales, table, zero, _i32(range(n + 1)), k.to(DEV), v.to(DEV))
    q = torch.full((1, 1, 1, D), 1.0)
    kd, vd = (_values(t[0][table.cpu().long()[0], w, 0].reshape(-1, D // 2)[: n + 1],
                      t[1][table.cpu().long()[0], w, 0].reshape(-1, D // 16)[: n + 1])
              for t, w in (((codes.cpu(), scales.cpu()), 0), ((codes.cpu(), scales.cpu()), 1)))
    score = float(q[0, 0, 0].double() @ kd[n])
    scale = 9.01 / score  # exp(9.01) = 8185: the two sides nearly balance
    got = cuda_lib.kv_attention(codes, scales, table, _i32([n]), q.to(DEV), scale=scale, dtype=F32)
    z = torch.cat((torch.zeros(n, dtype=torch.float64), torch.tensor([score * scale], dtype=torch.float64)))
    ref = torch.softmax(z, 0) @ vd
    # the two sides' weights are each off by at most 3 * 2^-11 * (1 + 9) in total
    assert torch.all((got.cpu()[0, 0, 0].double() - ref).abs() <= 30 * 2.0 ** -11 * vd.abs().amax())


def test_attention_invalid_pages_and_lengths(cuda_lib):
    B, T, H, kv, D, page = 4, 2, 4, 2, 64, 16
    codes, scales, table = _filled(cuda_lib, B, 4, kv, D, page, seed=31)
    table[0, 1] = -1        # a hole in the context
    table[1, 0] = 10 ** 6   # outside the pool
    table[3] = -5           # nothing at all
    lens = [40, 20, 1000, 30]  # the third is past its table: its drafted tokens have no place
    q = _rand(3, B, T, H, D, dtype=F16)
    ref, bar = _attention_ref(codes, scales, table, lens, q, None, D ** -0.5, F16)
    got = cuda_lib.kv_attention(codes, scales, table, _i32(lens), q.to(DEV))
    assert torch.all((got.cpu().double() - ref).norm(dim=-1) <= bar)
    assert not got[3].any()
    # a negative length is an empty context
    a = cuda_lib.kv_attention(codes, scales, table, _i32([0, 0, 0, 0]), q.to(DEV))
    b = cuda_lib.kv_attention(codes, scales, table, _i32([-3, -2 ** 31, 0, -1]), q.to(DEV))
    assert torch.equal(a, b)
    assert cuda_lib.kv_attention(codes, scales, table[:0], _i32([]), q[:0].to(DEV)).shape == (0, T, H, D)
    assert cuda_lib.kv_attention(codes, scales, table, _i32(lens), q[:, :0].to(DEV)).shape == (B, 0, H, D)


def test_attention_refuses_a_small_or_crooked_workspace(cuda_lib):
    codes, scales, table = _pool(cuda_lib, 2, 2, 2, 64, 16)
    q = torch.zeros(2, 3, 4, 64, device=DEV)
    need = cuda_lib.tq_kv_attention_workspace_bytes(2, 3, 4, 2, 64)
    ws = torch.empty(need + 256, dtype=torch.uint8, device=DEV)
    cuda_lib.kv_attention(codes, scales, table, _i32([1, 2]), q, ws=ws[:need])
    for bad in (ws[:need - 1], ws[8:]):
        with pytest.raises(cuda_lib.TQError, match="WORKSPACE"):
            cuda_lib.kv_attention(codes, scales, table, _i32([1, 2]), q, ws=bad)
    with pytest.raises(ValueError, match="lens"):
        cuda_lib.kv_attention(codes, scales, table, _i32([1, 2, 3]), q)
    with pytest.raises(ValueError, match="parents"):
        cuda_lib.kv_attention(codes, scales, table, _i32([1, 2]), q, parents=_i32([[0, 0]]))
    with pytest.raises(ValueError, match="q"):
        cuda_lib.kv_attention(codes, scales, table, _i32([1, 2]), q[:1])
    with pytest.raises(cuda_lib.TQError, match="ALIGNMENT"):
        cuda_lib.kv_attention(codes, scales, table, _i32([1, 2]), torch.zeros(2, 3, 4, 68, device=DEV)[..., 2:66])
    with pytest.raises(TypeError):
        cuda_lib.kv_attention(codes, scales, table, _i32([1, 2]), q.double())


def test_attention_rows_do_not_touch_one_another(cuda_lib):
    """NaN and infinity in one query row leave every other row's bits alone, on both kernels."""
    for T, H, kv in ((3, 4, 2), (16, 8, 2)):
        B, D, page = 2, 128, 16
        codes, scales, table = _filled(cuda_lib, B, 8, kv, D, page, seed=61)
        q, lens = _rand(2, B, T, H, D, dtype=BF16).to(DEV), _i32([70, 100])
        want = cuda_lib.kv_attention(codes, scales, table, lens, q)
        bad = q.clone()
        bad[0, 1, 2], bad[1, 2, 3, 5] = float("nan"), float("inf")
        got = cuda_lib.kv_attention(codes, scales, table, lens, bad)
        keep = torch.ones(B, T, H, dtype=torch.bool)
        keep[0, 1, 2] = keep[1, 2, 3] = False
        assert torch.equal(got.cpu()[keep], want.cpu()[keep])


def test_attention_reports_a_wait_that_runs_out(cuda_lib):
    """The tcgen05 kernel's bounded waits: keys that are never handed over end in a
    status, not in a hang, and the next call is right again."""
    B, T, H, kv, D, page = 2, 16, 8, 2, 128, 16
    codes, scales, table = _filled(cuda_lib, B, 20, kv, D, page, seed=71)
    q, lens = _rand(1, B, T, H, D, dtype=BF16).to(DEV), _i32([250, 300])
    ws = cuda_lib.kv_attention_workspace(B, T, H, kv, D)
    want = cuda_lib.kv_attention(codes, scales, table, lens, q, ws=ws)
    assert cuda_lib.workspace_status(ws) == 0
    cuda_lib.tq_debug_set_flags(32)
    try:
        cuda_lib.kv_attention(codes, scales, table, lens, q, ws=ws)
    finally:
        cuda_lib.tq_debug_set_flags(0)
    assert cuda_lib.workspace_status(ws, clear=False) == 8
    assert torch.equal(cuda_lib.kv_attention(codes, scales, table, lens, q, ws=ws), want)
    assert cuda_lib.workspace_status(ws) == 0


def test_attention_far_pages(cuda_lib):
    """Records beyond 2^32 bytes into the pool."""
    kv, D, page = 8, 128, 64
    pages = (1 << 32) // (2 * kv * page * D // 2) + 300
    codes = torch.empty(pages, 2, kv, page, D // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(pages, 2, kv, page, D // 16, dtype=torch.int16, device=DEV)
    near, nears, small = _filled(cuda_lib, 1, 4, kv, D, page, seed=41)
    far = torch.arange(pages - 4, pages, device=DEV)
    codes[far], scales[far] = near[small[0].long()], nears[small[0].long()]
    q = _rand(1, 1, 1, 32, D, dtype=BF16).to(DEV)
    a = cuda_lib.kv_attention(near, nears, small, _i32([222]), q)
    b = cuda_lib.kv_attention(codes, scales, far.to(torch.int32)[None].contiguous(), _i32([222]), q)
    assert torch.equal(a, b)
    zero, at = _i32([0] * 200), _i32(range(200))
    ka, va = cuda_lib.kv_read(near, nears, small, zero, at)
    kb, vb = cuda_lib.kv_read(codes, scales, far.to(torch.int32)[None].contiguous(), zero, at)
    assert torch.equal(ka, kb) and torch.equal(va, vb)


def test_attention_on_another_stream_and_in_graphs(cuda_lib):
    B, T, H, kv, D, page = 3, 4, 8, 2, 128, 16
    codes, scales, table = _filled(cuda_lib, B, 40, kv, D, page, seed=51)
    q, par = _rand(1, B, T, H, D, dtype=BF16).to(DEV), _tree(5, B, T).to(DEV)
    lens = _i32([100, 5, 600])
    want = cuda_lib.kv_attention(codes, scales, table, lens, q, parents=par)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = torch.empty_like(want)
    ws = cuda_lib.kv_attention_workspace(B, T, H, kv, D)
    cuda_lib.kv_attention(codes, scales, table, lens, q, parents=par, out=got, ws=ws, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    # two graphs that share a workspace, replayed in turn over lengths that change
    outs, graphs = [torch.empty_like(want) for _ in range(2)], []
    q2 = (q * 0.5).contiguous()
    with torch.cuda.stream(side):
        for out, query in zip(outs, (q, q2)):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                cuda_lib.kv_attention(codes, scales, table, lens, query, parents=par, out=out, ws=ws)
            graphs.append(g)
    torch.cuda.synchronize()
    for new in ([100, 5, 600], [0, 630, 17], [636, 1, 300]):
        lens.copy_(_i32(new))
        for g in graphs + graphs[:1]:
            g.replay()
        torch.cuda.synchronize()
        for out, query in zip(outs, (q, q2)):
            assert torch.equal(out, cuda_lib.kv_attention(codes, scales, table, lens, query, parents=par))


def test_attention_calls_at_once(cuda_lib):
    """Calls of both kernels on four streams that overlap, with workspaces of their own."""
    B, H, kv, D, page = 3, 8, 2, 128, 16
    codes, scales, table = _filled(cuda_lib, B, 60, kv, D, page, seed=53)
    lens = _i32([900, 5, 333])
    qs = [_rand(i, B, T, H, D, dtype=BF16).to(DEV) for i, T in enumerate((1, 30, 4, 20))]
    want = [cuda_lib.kv_attention(codes, scales, table, lens, q) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    got = [[] for _ in qs]
    for _ in range(20):
        for q, stream, outs in zip(qs, streams, got):
            outs.append(cuda_lib.kv_attention(codes, scales, table, lens, q, stream=stream))
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        assert all(torch.equal(o, w) for o in outs)


def test_what_a_call_allocates_belongs_to_its_stream(cuda_lib):
    # a call given a stream that is busy: memory that it allocated itself must not
    # be handed to later work of the current stream while the call still waits
    B, T, H, kv, D, page = 2, 3, 8, 2, 128, 16
    codes, scales, table = _filled(cuda_lib, B, 20, kv, D, page, seed=52)
    q, lens = _rand(1, B, T, H, D, dtype=BF16).to(DEV), _i32([300, 17])
    want = cuda_lib.kv_attention(codes, scales, table, lens, q)
    seqs, places = _i32([0, 1, 0]), _i32([5, 6, 299])
    want_k, want_v = cuda_lib.kv_read(codes, scales, table, seqs, places)
    nbytes = cuda_lib.tq_kv_attention_workspace_bytes(B, T, H, kv, D)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about 10 ms
    got = cuda_lib.kv_attention(codes, scales, table, lens, q, stream=side)
    got_k, got_v = cuda_lib.kv_read(codes, scales, table, seqs, places, stream=side)
    for _ in range(4):
        torch.zeros(nbytes, dtype=torch.uint8, device=DEV)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(got_k, want_k) and torch.equal(got_v, want_v)


# ---------------------------------------------------------------------------
# commit, and the whole step
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("layers,B,T,kv,dim,page", [(None, 1, 4, 1, 32, 16), (3, 5, 16, 2, 96, 16),
                                                    (2, 7, 64, 3, 128, 32), (1, 2, 64, 1, 256, 64)])
def test_commit(cuda_lib, layers, B, T, kv, dim, page):
    per = -(-T // page) + 2
    pages = B * per
    codes, scales = cuda_lib.kv_cache(pages, kv, dim, page, layers=layers)
    g = torch.Generator().manual_seed(T)
    codes.copy_(torch.randint(0, 256, codes.shape, generator=g).to(torch.uint8))
    scales.copy_(torch.randint(-30000, 30000, scales.shape, generator=g).to(torch.int16))
    table = torch.randperm(pages, generator=g).to(torch.int32).view(B, per).contiguous()
    lens = torch.randint(0, page + 1, (B,), generator=g).to(torch.int32)
    path = torch.full((B, T), -1, dtype=torch.int32)
    for b in range(B):
        count = [T, 0, 1, T // 2, T // 3, 2, T // 4][b % 7]
        path[b, :count] = torch.randperm(T, generator=g)[:count].sort().values.to(torch.int32)
    if B > 5:
        path[5, :4] = torch.tensor([3, 9, 9, 12])  # the branch ends where it does not increase
    want_c, want_s = codes.cpu().clone(), scales.cpu().clone()
    for t in (want_c, want_s):
        x = t if layers else t[None]
        for b in range(B):
            last = -1
            for i, src in enumerate(path[b].tolist()):
                if src <= last:
                    break
                last = src
                a, z = int(lens[b]) + src, int(lens[b]) + i
                if a // page < per:
                    x[:, table[b, z // page], :, :, z % page] = x[:, table[b, a // page], :, :, a % page]
    cuda_lib.kv_commit(codes, scales, table.to(DEV), lens.to(DEV), path.to(DEV))
    assert torch.equal(codes.cpu(), want_c) and torch.equal(scales.cpu(), want_s)


def test_commit_without_places(cuda_lib):
    codes, scales, table = _pool(cuda_lib, 3, 2, 1, 32, 16)
    codes.random_(0, 255)
    keep = codes.clone()
    table[0, 0] = -1
    path = _i32([[1, 3, 2 ** 31 - 1], [40, 50, 60], [0, 1, 2]])
    cuda_lib.kv_commit(codes, scales, table, _i32([0, 0, -7]), path)
    assert torch.equal(codes, keep)


def test_one_step_of_tree_decoding(cuda_lib):
    """Rotary positions, append, attention, commit over two layers as a decoder
    runs them: after the accepted branch is committed, the next token's attention
    equals that of a sequence which had decoded the branch token by token."""
    tq = cuda_lib
    layers, B, T, H, kv, D, page = 2, 2, 6, 8, 2, 128, 16
    codes, scales = tq.kv_cache(B * 8, kv, D, page, layers=layers)
    table = torch.arange(B * 8, dtype=torch.int32, device=DEV).view(B, 8)
    f = tq.rope_frequencies(D, 500000.0)
    lens = [37, 60]
    parents = torch.tensor([[-1, -1, 0, 1, 3, 3], [-1, 0, 0, 2, 1, 3]], dtype=torch.int32)
    branch = torch.tensor([[1, 3, 5], [0, 2, -1]], dtype=torch.int32)
    depth = torch.zeros(B, T, dtype=torch.int32)
    for b in range(B):
        for i in range(T):
            depth[b, i] = 0 if parents[b, i] < 0 else depth[b, parents[b, i]] + 1
    ctx_s = torch.cat([torch.full((n,), b) for b, n in enumerate(lens)])
    ctx_p = torch.cat([torch.arange(n) for n in lens])
    for layer in range(layers):
        k, v = _rand(layer, sum(lens), kv, D).to(DEV), _rand(layer + 9, sum(lens), kv, D).to(DEV)
        tq.kv_append(codes[layer], scales[layer], table, _i32(ctx_s), _i32(ctx_p), k, v, rope=(_i32(ctx_p), f))
    lens_d = _i32(lens)
    straight_c, straight_s = codes.clone(), scales.clone()  # the sequence decoded token by token
    seqs = torch.arange(B, dtype=torch.int32).repeat_interleave(T)
    places = (torch.tensor(lens)[:, None] + torch.arange(T)).to(torch.int32)
    pos = (torch.tensor(lens)[:, None] + depth).to(torch.int32).reshape(-1)
    for layer in range(layers):
        qkv = _rand(layer + 20, B * T, H + 2 * kv, D).to(DEV)  # as it leaves a fused projection
        q = tq.rope(qkv[:, :H], pos.to(DEV), f)
        k, v = qkv[:, H:H + kv], qkv[:, H + kv:]
        tq.kv_append(codes[layer], scales[layer], table, seqs.to(DEV), places.reshape(-1).to(DEV), k, v,
                     rope=(pos.to(DEV), f))
        out = tq.kv_attention(codes[layer], scales[layer], table, lens_d, q.view(B, T, H, D),
                              parents=parents.to(DEV), dtype=F32)
        for b in range(B):
            for i, t in enumerate(branch[b].tolist()):
                if t < 0:
                    break
                row = b * T + t
                tq.kv_append(straight_c[layer], straight_s[layer], table, _i32([b]), _i32([lens[b] + i]),
                             k[row:row + 1], v[row:row + 1], rope=(_i32([lens[b] + i]), f))
                alone = tq.kv_attention(straight_c[layer], straight_s[layer], table[b:b + 1], _i32([lens[b] + i]),
                                        q[row].view(1, 1, H, D), dtype=F32)
                # the same sums in another order and split
                assert (alone[0, 0] - out[b, t]).norm() <= 2e-3 * out[b, t].norm()
    tq.kv_commit(codes, scales, table, lens_d, branch.to(DEV))
    accepted = (branch >= 0).sum(1).to(torch.int32)
    after = lens_d + accepted.to(DEV)
    for layer in range(layers):
        q = _rand(layer + 40, B, 1, H, D).to(DEV)
        k, v = _rand(50, B, kv, D).to(DEV), _rand(51, B, kv, D).to(DEV)
        for c, s in ((codes, scales), (straight_c, straight_s)):
            tq.kv_append(c[layer], s[layer], table, _i32(range(B)), after, k, v, rope=(after, f))
        a = tq.kv_attention(codes[layer], scales[layer], table, after, q)
        b = tq.kv_attention(straight_c[layer], straight_s[layer], table, after, q)
        assert torch.equal(a, b)
