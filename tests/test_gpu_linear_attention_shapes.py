"""Linear attention over widths, types, head counts and lengths, each launch shape that they choose,
against the recurrence in fp64 on the GPU.

Tolerances as in test_gpu_linear_attention.py: u = 2^-24, h = 2^-8, A the same sums over absolute
values; a prompt or a token is off by c u A, c = T + d + d_v + 32, on the tensor cores (bf16) by
2^-16 A + h A more, and a bf16 result by h of itself.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from sparse_weight_memory_chunk_b200 import fwpkm  # noqa: E402

U, HB = 2.0 ** -24, 2.0 ** -8


def recurrence(q, k, v, ld, scale, s):
    q, k, v, s = (x.double() for x in (q, k, v, s))
    a = torch.exp(ld.double())[None, :, None, None]
    out = []
    for t in range(q.shape[2]):
        s = a * s + k[:, :, t, :, None] * v[:, :, t, None, :]
        out.append(scale * torch.einsum("bhd,bhde->bhe", q[:, :, t], s))
    return torch.stack(out, 2), s


def check(got, ref, size, c, bf16, what):
    tol = c * U * size
    if bf16:
        tol = tol + HB * (ref.abs() + tol)
    off = (got.double() - ref).abs()
    assert bool((off <= tol).all()), f"{what}: worst {float((off / tol).max()):.3g} of the bound"


@pytest.mark.parametrize("B,H,T", [(1, 1, 3), (2, 3, 20), (16, 16, 20), (10, 15, 40), (1, 2, 300)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [1, 7, 16, 33, 64, 72, 128, 200, 256])
def test_widths(B, H, T, dtype, d):
    bf = dtype == torch.bfloat16
    g = torch.Generator("cuda").manual_seed(1000 * d + T)
    ld = torch.tensor([(-0.03, -0.4, -6.0)[h % 3] for h in range(H)], device="cuda")
    for dv in (1, 12, 16, 37, 64, 100, 128, 256):
        q, k = (torch.randn(B, T, H, d, generator=g, device="cuda").to(dtype).transpose(1, 2) for _ in range(2))
        v = torch.randn(B, T, H, dv, generator=g, device="cuda").to(dtype).transpose(1, 2)
        s0 = torch.randn(B, H, d, dv, generator=g, device="cuda")
        ref, rs = recurrence(q, k, v, ld, 0.5, s0)
        size, as_ = recurrence(q.abs(), k.abs(), v.abs(), ld, 0.5, s0.abs())
        c = T + d + dv + 32
        co = c + (2.0 ** 16 + 2.0 ** 8 if bf else 0.0)
        what = f"d {d}, d_v {dv}"
        o, sT = fwpkm.linear_attention(q, k, v, ld, scale=0.5, s0=s0, final_state=True)
        check(o, ref, size, co, bf, f"{what}: o")
        check(sT, rs, as_, c, False, f"{what}: sT")
        if T <= 20:
            o, sT = fwpkm.linear_attention_step(q, k, v, ld, s0, scale=0.5, in_place=False)
            check(o, ref, size, c, bf, f"{what}: o by step")
            check(sT, rs, as_, c, False, f"{what}: state by step")
    fwpkm.linear_attention_sync()
