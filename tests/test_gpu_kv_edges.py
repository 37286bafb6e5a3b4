"""GPU checks of the key/value cache operators at their edges: chains with the
products, scores and values of extreme size, queries that are not finite.
References and bars: test_gpu_kv_cache.py."""
import pytest
import torch

from test_gpu_kv_cache import BF16, DEV, F16, F32, _attention_ref, _filled, _forward, _i32, _rand, _rotated_domain

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# chains
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("rows", [1, 4, 16, 32, 40])
def test_products_of_what_the_kernel_before_writes(cuda_lib, rows):
    """rope and kv_attention into the products, one stream, no wait between, inputs
    that change and outputs in the same memory every time: the same bits as with a
    wait after every call."""
    tq = cuda_lib
    H, kv, D, page, n = 8, 2, 128, 16, 512
    B, T = (rows, 1) if rows < 8 else (rows // 4, 4)
    codes, scales, table = _filled(tq, B, 4, kv, D, page, seed=rows)
    lens = _i32([(7 * b) % 60 for b in range(B)])
    w = _rand(3, n, H * D, dtype=BF16).to(DEV)
    wc, ws = tq.quantize(w)
    nc, ns, nt = tq.nvfp4_quantize(w)
    f, pos = tq.rope_frequencies(D), _i32(range(rows))
    qs = [_rand(10 + i, rows, H, D, dtype=BF16).to(DEV) for i in range(12)]
    work, aws = tq.workspace(rows, n, H * D), tq.kv_attention_workspace(B, T, H, kv, D)  # no launch between the calls
    x, o = torch.empty_like(qs[0]), torch.empty(B, T, H, D, dtype=BF16, device=DEV)

    def step(q, wait):
        tq.rope(q, pos, f, out=x)
        wait()
        y = [tq.gemm(wc, ws, n, H * D, x.view(rows, -1), ws=work)]
        wait()
        tq.kv_attention(codes, scales, table, lens, x.view(B, T, H, D), out=o, ws=aws)
        wait()
        y.append(tq.gemm(wc, ws, n, H * D, o.view(rows, -1), ws=work))
        wait()
        tq.rope(o.view(rows, H, D), pos, f, out=x)
        wait()
        if rows <= 32:
            y.append(tq.nvfp4_gemm(nc, ns, nt, n, H * D, x.view(rows, -1), ws=work))
            wait()
        return y

    want = [step(q, torch.cuda.synchronize) for q in qs]
    for _ in range(5):
        got = [step(q, lambda: None) for q in qs]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(s, t) for s, t in zip(a, b))


# ---------------------------------------------------------------------------
# scores, values and queries of extreme size
# ---------------------------------------------------------------------------
def _rows(codes, scales, table, lens, q):
    """Per row of a chain: rotated query, the records that it sees (keys, values),
    all in the rotated domain and fp64."""
    B, T, H, D = q.shape
    kv, page = codes.shape[2], codes.shape[3]
    table, codes, scales = table.cpu().long(), codes.cpu(), scales.cpu()
    qr = _forward(q) / 32
    for b in range(B):
        place = torch.arange(int(lens[b]) + T)
        at = table[b, place // page]
        for h in range(kv):
            k, v = (_rotated_domain(codes[at, w, h, place % page], scales[at, w, h, place % page]) for w in (0, 1))
            for t in range(T):
                n = int(lens[b]) + t + 1
                for g in range(H // kv):
                    yield (b, t, h * (H // kv) + g), qr[b, t, h * (H // kv) + g], k[:n], v[:n]


# (rows of a key/value head: 4 and 12 on mma.sync, 64 and 160 on tcgen05)
@pytest.mark.parametrize("T,H,kv,D", [(1, 4, 1, 128), (3, 8, 2, 64), (2, 4, 2, 256), (16, 8, 2, 128), (40, 8, 2, 64)])
@pytest.mark.parametrize("size", [100.0, 1000.0, 60000.0 / 4])
def test_attention_with_the_largest_scale(cuda_lib, T, H, kv, D, size):
    """|scale| = 65536, the documented limit: scores up to 2^40 times log2(e).  The weights
    stay finite, one token has all of the weight, and its value comes out."""
    lens = [300, 77]
    codes, scales, table = _filled(cuda_lib, 2, 22, kv, D, 16, seed=81)
    q = _rand(7, 2, T, H, D, dtype=BF16, scale=size).clamp(-60000, 60000)
    for scale in (65536.0, -65536.0):
        got = cuda_lib.kv_attention(codes, scales, table, _i32(lens), q.to(DEV), scale=scale, dtype=F32).cpu().double()
        assert torch.all(torch.isfinite(got))
        clear = 0
        for row, x, k, v in _rows(codes, scales, table, lens, q):
            z = k @ x * scale
            top = z.topk(2).values
            # scores are off by 2^-11 of the products' 2-norm rms; eight times that on each side, and weights
            # of the others below e^-60
            if top[0] - top[1] < 16 * 2.0 ** -11 * (k * x).norm(dim=1).amax() * abs(scale) + 60:
                continue
            clear += 1
            best = v[z.argmax()]
            out = _forward(got[row][None])[0]  # H (s . out) = the rotated value
            assert (out - best).norm() <= 3 * 2.0 ** -11 * best.norm(), row
        assert clear > T * H  # of 2 T H rows


@pytest.mark.parametrize("T,H,kv,D", [(1, 4, 1, 128), (3, 8, 2, 96), (2, 4, 2, 256), (16, 8, 2, 128), (40, 8, 2, 64)])
@pytest.mark.parametrize("size,scale", [(1e-5, 65536.0), (1e-6, 65536.0), (1e-6, -3e4), (1e-9, 65536.0),
                                        (3e4, 1e-4), (1e-7, 0.0)])
def test_attention_with_queries_of_any_size(cuda_lib, T, H, kv, D, size, scale):
    """Small queries keep their bits (fp16 alone has steps of 2^-24 there), large ones stay finite."""
    lens = [200, 31]
    codes, scales, table = _filled(cuda_lib, 2, 16, kv, D, 16, seed=83)
    q = _rand(8, 2, T, H, D, scale=size)
    q[:, :, 0] *= 2.0 ** -7  # rows of one tile that are far apart
    got = cuda_lib.kv_attention(codes, scales, table, _i32(lens), q.to(DEV), scale=scale, dtype=F32)
    ref, bar = _attention_ref(codes, scales, table, lens, q, None, scale, F32)
    assert torch.all((got.cpu().double() - ref).norm(dim=-1) <= bar)


@pytest.mark.parametrize("T,H,kv,D", [(1, 4, 1, 128), (2, 4, 2, 256), (16, 8, 2, 128), (40, 8, 2, 64)])
@pytest.mark.parametrize("size,scale", [(1e-4, 1e3), (1e-5, 1e4), (1e-6, 65536.0)])
def test_attention_over_small_records(cuda_lib, T, H, kv, D, size, scale):
    """Keys and values so small that centroid times scale is subnormal in fp16: each
    product is rounded to a multiple of 2^-24, off by 2^-24 / sqrt(12) rms.  Beside
    the usual bar that is a score off by |q'| scale times it, and a row off by
    sqrt(sum p_j^2) sqrt(D / 32) times it; again four times the rms."""
    lens, page, per = [200, 31], 16, 16
    codes, scales, table = cuda_lib.kv_cache(2 * per, kv, D, page) + (_i32(range(2 * per)).view(2, per),)
    n = per * page
    seqs, places = _i32(torch.arange(2).repeat_interleave(n)), _i32(torch.arange(n).repeat(2))
    k, v = _rand(91, 2 * n, kv, D, scale=size), _rand(92, 2 * n, kv, D, scale=size)
    cuda_lib.kv_append(codes, scales, table, seqs, places, k.to(DEV), v.to(DEV))
    q = _rand(9, 2, T, H, D)
    got = cuda_lib.kv_attention(codes, scales, table, _i32(lens), q.to(DEV), scale=scale, dtype=F32).cpu().double()
    ref, bar = _attention_ref(codes, scales, table, lens, q, None, scale, F32)
    step = 2.0 ** -24 / 12 ** 0.5
    for row, x, kk, vv in _rows(codes, scales, table, lens, q):
        p = torch.softmax(kk @ x * scale, 0)
        spread = (p.square() * vv.square().sum(1) / 32).sum().sqrt()
        floor = step * (x.norm() * scale * spread + p.norm() * (D / 32) ** 0.5)
        assert (got[row] - ref[row]).norm() <= bar[row] + 4 * floor, row


@pytest.mark.parametrize("T,H,kv,D", [(1, 4, 1, 128), (3, 8, 2, 96), (4, 2, 1, 256), (16, 8, 2, 128), (40, 8, 2, 64)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_queries_that_are_not_finite_answer_nan(cuda_lib, T, H, kv, D, dtype):
    """A NaN, an infinity or an overflow upstream does not turn into a plausible row;
    other rows keep their bits, and a row without a token still answers zeros."""
    B = 3
    codes, scales, table = _filled(cuda_lib, B, 22, kv, D, 16, seed=85)
    table[2] = -1  # nothing to attend to
    lens = _i32([300, 1, 100])
    q = _rand(7, B, T, H, D, dtype=dtype).to(DEV)
    want = cuda_lib.kv_attention(codes, scales, table, lens, q)
    assert torch.all(torch.isfinite(want)) and not want[2].any()
    bad, hit = q.clone(), torch.zeros(B, T, H, dtype=torch.bool, device=DEV)
    values = [float("nan"), float("inf"), -float("inf")] + ([3e38, -1e38] if dtype != F16 else [])
    at = [(b, t, h, e) for b in range(B) for t, h, e in ((0, 1, 5), (T - 1, H - 1, D - 1), (T // 2, 0, 0))]
    for i, (b, t, h, e) in enumerate(at):
        bad[b, t, h, e] = values[i % len(values)]
        hit[b, t, h] = True
    bad[0, 0, 1] = float("inf")  # a whole row
    for scale in (None, -1.0):
        want = cuda_lib.kv_attention(codes, scales, table, lens, q, scale=scale)
        got = cuda_lib.kv_attention(codes, scales, table, lens, bad, scale=scale)
        assert torch.all(torch.isnan(got[:2][hit[:2]]))
        assert torch.equal(got[~hit], want[~hit])
        assert not got[2].any()
    # a drafted token that is not there answers zeros, whatever its query holds
    if T > 1:
        parents = torch.arange(-1, T - 1, dtype=torch.int32).repeat(B, 1)
        parents[:, T - 1] = -2
        got = cuda_lib.kv_attention(codes, scales, table, lens, bad, parents=parents.to(DEV))
        assert not got[:, T - 1].any()


@pytest.mark.parametrize("T,H,kv,D", [(1, 4, 1, 128), (16, 8, 2, 128), (40, 8, 2, 64)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_queries_near_the_types_limit(cuda_lib, T, H, kv, D, dtype):
    """With a scale as small as the queries are large: right up to 2^121, NaN where the sum
    of a block's 32 elements may overflow (all scores minus infinity are no empty row)."""
    codes, scales, table = _filled(cuda_lib, 1, 22, kv, D, 16, seed=87)
    lens = [0]
    q = _rand(7, 1, T, H, D, dtype=F32).clamp(-2, 2).to(dtype)
    ref, bar = _attention_ref(codes, scales, table, lens, q, None, 0.5, F32)
    got = cuda_lib.kv_attention(codes, scales, table, _i32(lens), (q.float() * 2.0 ** 120).to(dtype).to(DEV),
                                scale=2.0 ** -121, dtype=F32)
    assert torch.all((got.cpu().double() - ref).norm(dim=-1) <= bar)
    signs = torch.where(_rand(8, 1, T, H, D) < 0, -1.0, 1.0)
    for value in (2.0 ** 122, 3e38):
        for sign in (1.0, -1.0, signs):
            far = (torch.full((1, T, H, D), value) * sign).to(dtype).to(DEV)
            assert torch.all(torch.isnan(cuda_lib.kv_attention(codes, scales, table, _i32(lens), far, scale=2.0 ** -121)))


# ---------------------------------------------------------------------------
# status
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T,H,kv,D", [(16, 8, 2, 128), (40, 8, 2, 64)])
def test_attention_reports_of_every_cta_count(cuda_lib, T, H, kv, D):
    """What a CTA of the tcgen05 kernel reports at its start is not lost to the word being
    cleared by another one, whichever of them comes first."""
    B, page = 40, 16
    codes, scales, table = _filled(cuda_lib, B, 20, kv, D, page, seed=73)
    q, lens = _rand(1, B, T, H, D, dtype=BF16).to(DEV), _i32([(37 * b) % 250 for b in range(B)])
    ws = cuda_lib.kv_attention_workspace(B, T, H, kv, D).fill_(255)
    want = cuda_lib.kv_attention(codes, scales, table, lens, q, ws=ws)
    assert cuda_lib.workspace_status(ws) == 0
    for _ in range(20):
        cuda_lib.tq_debug_set_flags(64)
        try:
            cuda_lib.kv_attention(codes, scales, table, lens, q, ws=ws)
        finally:
            cuda_lib.tq_debug_set_flags(0)
        assert cuda_lib.workspace_status(ws, clear=False) == 8
        assert torch.equal(cuda_lib.kv_attention(codes, scales, table, lens, q, ws=ws), want)
        assert cuda_lib.workspace_status(ws, clear=False) == 0


# ---------------------------------------------------------------------------
# types
# ---------------------------------------------------------------------------
def test_read_and_attention_take_the_outputs_type(cuda_lib):
    codes, scales, table = _filled(cuda_lib, 1, 2, 2, 64, 16, seed=3)
    zero, at = _i32([0, 0]), _i32([3, 17])
    want, _ = cuda_lib.kv_read(codes, scales, table, zero, at, dtype=F32)
    k, v = cuda_lib.kv_read(codes, scales, table, zero, at)
    assert k.dtype == v.dtype == BF16 and torch.equal(k, want.to(BF16))
    given = torch.empty(2, 2, 64, dtype=F16, device=DEV)
    k, v = cuda_lib.kv_read(codes, scales, table, zero, at, k=given)
    assert k is given and v.dtype == F16 and torch.equal(k, want.half())
    q, out = _rand(1, 1, 1, 4, 64, dtype=BF16).to(DEV), torch.empty(1, 1, 4, 64, device=DEV)
    assert cuda_lib.kv_attention(codes, scales, table, _i32([20]), q, out=out) is out
    assert torch.equal(out, cuda_lib.kv_attention(codes, scales, table, _i32([20]), q, dtype=F32))


# ---------------------------------------------------------------------------
# the largest sizes, and calls captured together
# ---------------------------------------------------------------------------
def _chain_ref(codes, scales, table, lens, q, scale, out_dtype):
    """_attention_ref of a chain, all rows of a (sequence, head) at once, on the GPU."""
    B, T, H, D = q.shape
    kv, page = codes.shape[2], codes.shape[3]
    G = H // kv
    q = q.cpu()
    qr = (_forward(q) / 32).to(DEV)
    ref, bar = torch.zeros(B, T, H, D, device=DEV, dtype=torch.float64), torch.zeros(B, T, H, device=DEV, dtype=torch.float64)
    table_h, codes_h, scales_h = table.cpu().long(), codes.cpu(), scales.cpu()
    for b in range(B):
        n = int(lens[b]) + T
        place = torch.arange(n)
        at = table_h[b, place // page]
        hidden = torch.arange(n)[None] > int(lens[b]) + torch.arange(T)[:, None]
        hidden = hidden.repeat_interleave(G, 0).to(DEV)
        for h in range(kv):
            k, v = (_rotated_domain(codes_h[at, w, h, place % page], scales_h[at, w, h, place % page]).to(DEV)
                    for w in (0, 1))
            x = qr[b, :, h * G:(h + 1) * G].reshape(T * G, D)
            p = torch.softmax((x @ k.T * scale).masked_fill(hidden, -torch.inf), 1)
            s = (x.square() @ k.square().T).masked_fill(hidden, 0).amax(1).sqrt() * abs(scale)
            o = _forward((p @ v).cpu()).to(DEV) / 32  # H (s . y); H y with the signs behind has the same norm
            spread = (p.square() @ (v.square().sum(1) / 32)).sqrt()
            ref[b, :, h * G:(h + 1) * G] = (p @ v).view(T, G, D)
            bar[b, :, h * G:(h + 1) * G] = (4 * 2.0 ** -11 * (1 + s) * spread
                                            + torch.finfo(out_dtype).eps / 2 * o.norm(dim=1)).view(T, G)
    return ref, bar


@pytest.mark.parametrize("B,T,H,kv,D,lens", [
    (1, 2, 1024, 1, 64, [70]),      # 2048 rows of one head, tcgen05
    (1, 2, 1024, 1, 32, [70]),      # the same on mma.sync
    (1, 64, 1024, 1, 64, [40]),     # 65536 rows
    (1, 1, 1024, 1024, 32, [33]),   # as many key/value heads
    (4096, 1, 1, 1, 32, None),      # as many sequences, mma.sync
    (4096, 17, 1, 1, 64, None),     # and tcgen05
])
def test_attention_at_the_largest_sizes(cuda_lib, B, T, H, kv, D, lens):
    lens = [(7 * b) % 30 for b in range(B)] if lens is None else lens
    codes, scales, table = _filled(cuda_lib, B, -(-(max(lens) + T) // 16), kv, D, 16, seed=D)
    q = _rand(H, B, T, H, D, dtype=F16)
    got = cuda_lib.kv_attention(codes, scales, table, _i32(lens), q.to(DEV), scale=0.25, dtype=F32)
    some = list(range(B)) if B < 100 else [0, 1, 2, 29, 500, 1023, 1024, 2047, 4094, 4095]
    ref, bar = _chain_ref(codes, scales, table[some], [lens[b] for b in some], q[some], 0.25, F32)
    turned = _forward(got[some].cpu()).to(DEV)  # H (s . out): the rotated domain, whose norm is sqrt(32) times larger
    assert torch.all((turned - ref).norm(dim=-1) / 32 ** 0.5 <= bar)


def test_graphs_of_both_kernels_share_a_workspace(cuda_lib):
    """Captured calls of one token and of a tree, one workspace, replayed in turn, over lengths
    and pages that change between replays."""
    tq = cuda_lib
    B, H, kv, D, page = 3, 8, 2, 128, 16
    codes, scales, table = _filled(tq, B, 40, kv, D, page, seed=57)
    lens = _i32([100, 5, 600])
    qs = [_rand(i, B, T, H, D, dtype=BF16).to(DEV) for i, T in enumerate((1, 30, 5, 64))]
    nbytes = max(tq.kv_attention_workspace(B, q.shape[1], H, kv, D).numel() for q in qs)
    ws = torch.full((nbytes,), 255, dtype=torch.uint8, device=DEV)
    outs, graphs, side = [torch.empty_like(q) for q in qs], [], torch.cuda.Stream()
    for q, out in zip(qs, outs):  # (kernels are loaded before the capture)
        tq.kv_attention(codes, scales, table, lens, q, out=out, ws=ws)
    torch.cuda.synchronize()
    for q, out in zip(qs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            tq.kv_attention(codes, scales, table, lens, q, out=out, ws=ws)
        graphs.append(g)
    order = torch.arange(B * 40, dtype=torch.int32).view(B, 40)
    for step, new in enumerate(([100, 5, 570], [0, 576, 17], [576, 1, 300])):
        lens.copy_(_i32(new))
        table.copy_(order.roll(step, 0))
        for _ in range(3):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        assert tq.workspace_status(ws) == 0
        for q, out in zip(qs, outs):
            assert torch.equal(out, tq.kv_attention(codes, scales, table, lens, q))
