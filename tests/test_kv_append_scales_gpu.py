"""The e4m3 append at the ends of the scales' range: a value of 0 gets code 0
whatever the scale, and no finite value a NaN."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [0.0, 1e-45, 1e-40, 2.0 ** -127, 2.0 ** -126, 1e-30, 1.0, 1e30, 3e38])
def test_codes_of_all_sizes(scale):
    import bf16_causal_prefill_02_b200 as zq

    x = torch.tensor([0.0, -0.0, 1e-40, -1e-38, 1e-37, 1e-30, 1.0, -3.0, 1e20, 3e38], dtype=torch.bfloat16)
    k = torch.zeros((1, 1, 128), dtype=torch.bfloat16)
    k[0, 0, :10] = x
    ds = torch.tensor([scale], device="cuda")
    kc, vc = (torch.full((1, 16, 1, 128), 0x7F, dtype=torch.uint8, device="cuda") for _ in "kv")
    zq.kv_append(k.cuda(), k.cuda(), kc, vc, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"),
                 k_descale=ds, v_descale=ds)
    inv = 0.0 if scale == 0.0 else (1.0 / ds.cpu()).clamp(max=torch.finfo(torch.float32).max)
    want = (k[0, 0].float() * inv).clamp(-448, 448).to(torch.float8_e4m3fn).float()
    for c in (kc, vc):
        assert torch.equal(c[0, 0, 0].view(torch.float8_e4m3fn).float().cpu(), want)
