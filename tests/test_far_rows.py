"""Gated experts, block norms and orthogonalised updates on rows whose offsets
pass 32 bits: the same bits as on dense copies."""
import pytest
import torch

import dnn_conv2d_bwd_amd as cbd

TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
FAR = 1 << 22  # elements between rows: 256 of them in bf16 are 2 GiB


def far(t, pitch):
    """t's rows in a buffer of `pitch` elements a row."""
    buf = torch.empty(t.shape[0] * pitch, dtype=t.dtype, device="cuda")
    v = buf.view(t.shape[0], pitch)[:, :t.shape[1]]
    v.copy_(t)
    assert (t.shape[0] - 1) * pitch > 2 ** 31
    return v


def same(got, want):
    for i, (a, b) in enumerate(zip(got, want)):
        assert (a is None and b is None) or torch.equal(a, b), f"result {i}"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kernel,pitch", [("bf16", "AUTO", FAR - 256), ("bf16", "STREAM", FAR - 256),
                                                ("f32", "AUTO", FAR // 2 - 256)])
def test_gated(dtype, kernel, pitch):
    """More rows than 2^31 / pitch, on three experts; 256 of them stay below 2 GiB."""
    print("[far] gated", dtype, kernel, flush=True)
    t, c, k = 2 ** 31 // pitch + 90, 64, 128
    gen = torch.Generator("cuda").manual_seed(1)
    draw = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(TORCH[dtype])
    x, w, down, dy = draw(t, c), draw(3, 2 * k, c) / 8, draw(3, c, k) / 11, draw(t, c)
    ends = torch.tensor([200, 300, t - 5], dtype=torch.int32, device="cuda")
    p = cbd.expert_plan(t, 3, c, 2 * k, dtype=dtype, force_kernel=getattr(cbd, f"EXPERT_KERNEL_{kernel}"))
    d = cbd.expert_plan(t, 3, k, c, dtype=dtype)
    h, gu, dgu = (torch.zeros(t, n, dtype=TORCH[dtype], device="cuda") for n in (k, 2 * k, 2 * k))
    cbd.expert_gated_forward(p, x, w, ends, h=h, gu=gu)
    cbd.expert_gated_bwd(d, dy, down, gu, ends, dgu=dgu)
    fx, fdy, fh, fgu, fdgu = (far(v, pitch) for v in (x, dy, torch.zeros_like(h), torch.zeros_like(gu), torch.zeros_like(gu)))
    cbd.expert_gated_forward(p, fx, w, ends, h=fh, gu=fgu)
    cbd.expert_gated_bwd(d, fdy, down, fgu, ends, dgu=fdgu)
    same((fh, fgu, fdgu), (h, gu, dgu))
    assert h[:t - 5].abs().sum(1).min() > 0 and not h[t - 5:].any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,c", [("bf16", 200), ("f32", 515), ("bf16", 9000)])
def test_block(dtype, c):
    print("[far] block", dtype, c, flush=True)
    pitch, t = FAR, 2 ** 31 // FAR + 20
    gen = torch.Generator("cuda").manual_seed(2)
    draw = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(TORCH[dtype])
    rows = [draw(t, c) for _ in range(5)]
    a, b = draw(c), draw(c)
    p = cbd.block_plan(t, c, dtype)

    def run(r, y, g, dz, dn, out):
        kw = dict(w_post=a, gate=g, w_pre=b)
        z, n, stats = cbd.block_forward(p, r, y, save=True, z=out(), n=out(), **kw)
        return (z, n, stats, *cbd.block_bwd(p, dz, dn, r, y, stats, dr=out(), dy=out(), dgate=out(), **kw))

    want = run(*rows, lambda: None)
    got = run(*(far(v, pitch) for v in rows), lambda: far(torch.zeros_like(rows[0]), pitch))
    same(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,shape", [("bf16", (3, 70, 96)), ("f32", (2, 200, 100)), ("bf16", (2, 40, 2100))])
def test_updates(dtype, shape):
    """Matrices 2^31 elements apart."""
    print("[far] updates", dtype, shape, flush=True)
    n, r, c = shape
    m = (torch.randn(shape, generator=torch.Generator().manual_seed(3)) / 30).to(TORCH[dtype]).cuda()
    apart = 2 ** 31 + 64
    far_m, far_out = (torch.empty((n - 1) * apart + r * c, dtype=m.dtype, device="cuda").as_strided(shape, (apart, c, 1))
                      for _ in range(2))
    far_m.copy_(m)
    p = cbd.ortho_plan(*shape, dtype=dtype, steps=3)
    want = cbd.orthogonalize(p, m)
    same((cbd.orthogonalize(p, far_m, far_out),), (want,))
    assert float(want.float().norm()) > 1
