"""moe_group_product where a workgroup of the streaming kernel takes a run of
2, 3 or 4 tiles of 64 weight rows: every output against the float64 product."""
import pytest

from tests.test_gpu_product import _sizes

pytestmark = pytest.mark.gpu

MAGS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _values(codes, scales):
    """float64 values of MXFP4 rows on the device."""
    import torch
    table = torch.tensor(MAGS + tuple(-m for m in MAGS), dtype=torch.float64, device=codes.device)
    v = table[torch.stack((codes & 15, codes >> 4), -1).to(torch.int32)].reshape(*scales.shape, 32)
    return (v * torch.exp2(scales.double() - 127.0)[..., None]).reshape(codes.shape[0], -1)


def _tiles(G, M, N):
    """Tiles of 64 weight rows a workgroup takes: what makes 4096 workgroups, at most 4."""
    return max(1, min(4, -(-N // 64) * min(G + M // 16, M) // 4096))


# widths off every multiple of 64; odd and even numbers of scale blocks; k past what fits LDS at once (4608)
@pytest.mark.parametrize("G,M,N,K,tiles,f32,gathered", [
    (300, 700, 1603, 544, 2, True, False), (300, 700, 2301, 1152, 3, False, True),
    (300, 700, 3170, 352, 4, True, True), (384, 512, 2600, 1216, 4, True, False),
    (384, 1536, 2700, 288, 4, False, False),
    (64, 600, 5190, 4640, 2, True, False), (64, 600, 10370, 4672, 4, False, True)])
def test_runs_of_tiles(gpu_lib, G, M, N, K, tiles, f32, gathered):
    import numpy as np
    import torch
    assert _tiles(G, M, N) == tiles and M <= 10 * G
    gen = torch.Generator(device="cuda").manual_seed(N + K)
    byte = lambda lo, hi, *s: torch.randint(lo, hi, s, dtype=torch.uint8, device="cuda", generator=gen)  # noqa: E731
    T = M // 4 if gathered else M
    a, a_sc = byte(0, 256, T, K // 2), byte(120, 126, T, K // 32)
    w, w_sc = byte(0, 256, G, N, K // 2), byte(120, 126, G, N, K // 32)
    sizes = _sizes(np.random.default_rng(N), G, M, "uneven")
    assert sizes.max() > 16                       # a group of more than one row tile too
    at = np.concatenate([[0], np.cumsum(sizes)])
    ids = torch.randperm(M, generator=gen, device="cuda").to(torch.int32) if gathered else None
    src = torch.arange(M, device="cuda") if ids is None else ids.long() // 4
    out = torch.full((M, N), float("nan"), dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    gpu_lib.group_product("mxfp4", a, a_sc, w, w_sc, torch.from_numpy(at.astype(np.int32)).cuda(), out, row_ids=ids,
                          id_div=4)
    av = _values(a, a_sc)
    for g in range(G):
        lo, hi = int(at[g]), int(at[g + 1])
        if lo == hi:
            continue
        rows, wv = av[src[lo:hi]], _values(w[g], w_sc[g])
        ref, size = rows @ wv.t(), rows.abs() @ wv.abs().t()
        # products of codes are exact, sums are fp32 (one rounding per 128 of k and lane group); bf16: half an ulp
        tol = (K / 128 + 8) * 2.0 ** -22 * size + (0 if f32 else 2.0 ** -8 * ref.abs())
        assert bool(((out[lo:hi].double() - ref).abs() <= tol).all()), g
