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
