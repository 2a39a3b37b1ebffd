"""The 8-bit form's codes and scales bit for bit: the scale is max|x| / 448 and the code the e4m3 value nearest to x / scale,
both quotients rounded to float32, ties to even.  Nothing is left to a tolerance: half of the cases in which a product
with 1 / scale gives another code are exact ties."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")


def form(x):
    """(codes as bytes, scales) of [rows, dim] on the CPU, from numpy's float32 quotients."""
    x = x.float().cpu().numpy()
    dim = x.shape[-1]
    y = np.pad(x, ((0, 0), (0, -dim % 128))).reshape(len(x), -1, 128)
    top = np.abs(y).max(-1)
    scale = np.where(top > 0, np.maximum(top / np.float32(448), np.float32(2.0 ** -126)), np.float32(1)).astype(np.float32)
    q = (y / scale[..., None]).astype(np.float32).reshape(len(x), -1)[:, :dim]
    return torch.from_numpy(np.ascontiguousarray(q)).to(torch.float8_e4m3fn).view(torch.uint8), torch.from_numpy(scale)


def check(x):
    import selective_state_space_41_amd as V
    codes, scale = V.act8_pack(x)
    want, ws = form(x)
    assert torch.equal(scale.cpu(), ws)
    off = codes.view(torch.uint8).cpu() != want
    assert not off.any(), f"{int(off.sum())} of {off.numel()} codes are not the nearest"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,dim", [(1, 1), (3000, 768), (4000, 130), (700, 2051), (9000, 72)])
def test_every_code_is_the_nearest(rows, dim, dtype):
    gen = torch.Generator(device="cuda").manual_seed(rows + dim)
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    check((normal(rows, dim) * (0.2 + normal(dim).abs())).to(dtype))


@pytest.mark.parametrize("exponent", [-149, -130, -126, -118, -100, 0, 100, 118])
def test_small_and_large_groups(exponent):
    """Scales down to the smallest normal number and below (where it stands for them), and near the largest."""
    gen = torch.Generator(device="cuda").manual_seed(exponent + 200)
    x = torch.randn(300, 200, generator=gen, device="cuda", dtype=torch.float64).clamp(-3.9, 3.9) * 2.0 ** exponent
    check(x.float())
    check(x.bfloat16())


def test_ties_go_to_the_even_code():
    """Whole numbers under a scale of 1 and of 3: 17 lies between the codes 16 and 18, 19 between 18 and 20, and so on."""
    x = torch.arange(-448, 449, device="cuda").float().reshape(-1, 1).expand(-1, 128).clone()
    x[:, 5] = 448.0
    for t in (x, 3 * x):
        check(t)
        check(t.bfloat16())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_zeros_keep_their_signs(dtype):
    x = torch.randn(4, 256, device="cuda").to(dtype)
    x[0, ::3], x[1, ::2], x[2] = -0.0, 0.0, -0.0
    check(x)


def test_all_bfloat16_values_under_all_scales():
    """Every significand of a group's largest magnitude with every significand of a value, over the codes' whole range."""
    top = torch.arange(128, 256, device="cuda").float()[:, None, None] * 2.0 ** -7
    value = torch.arange(128, 256, device="cuda").float()
    x = value[None, None, :127].expand(128, 20, 127) * 2.0 ** -torch.arange(7, 27, device="cuda").float()[None, :, None]
    x = torch.cat([torch.minimum(x, top), top.expand(128, 20, 1)], -1).reshape(-1, 128)
    y = torch.cat([torch.minimum(value[1:128].expand(2560, 127) * 2.0 ** -9, x[:, 127:]), x[:, 127:]], -1)
    for t in (x, y):
        assert torch.equal(t.bfloat16().float(), t)
        check(t.bfloat16())
        check(t)
