"""GPU: the example's mixture-of-experts layer against float64 on the same
quantised weights.

int8 rounds each activation to within 1/254 of its row's largest value; with
rows of a few hundred normal values (largest about 3.5 times the root mean
square) that is a relative error of about 3.5 / 127 / sqrt(12) = 0.8% per
rounding, twice in the layer, and the bf16 intermediates add less; MXFP4 (a
grid of 8 magnitudes: up to 1/6 of a value, about 7-10% in the mean square)
rounds the same two tensors, and its activations also to int8.  The bounds
leave a factor of two."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_layer  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("fmt,bound", [("w8a8", 0.03), ("mxfp4", 0.3)])
@pytest.mark.parametrize("T", [1, 7, 150])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_layer(fmt, bound, T, dtype):
    print("[case] layer", fmt, T, dtype, flush=True)
    layer = moe_layer.random_layer(12, 512, 288, 3, fmt, dtype, seed=T)
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, 512, generator=g, device="cuda").to(dtype)
    r = torch.randn(T, 512, generator=g, device="cuda").to(dtype)
    out, h = layer(x, r)
    ref, href = layer.plain(x, r)
    assert out.dtype == dtype and torch.equal(h, href)
    assert ((out.double() - ref).norm() / ref.norm()).item() < bound


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_routing_changes(dtype):
    """None where the experts' logits lie far apart; two of three where the
    choices share one; else what a plain loop over float64 logits counts."""
    layer = moe_layer.random_layer(12, 512, 32, 3, "w8a8", dtype, seed=1)
    g = torch.Generator(device="cuda").manual_seed(2)
    r = torch.zeros(200, 512, device="cuda", dtype=dtype)
    # token t is made of the rows of experts t, t + 1 and t + 2, in falling parts
    e = torch.eye(12, device="cuda").double()
    part = 4 * e + 3 * e.roll(1, 1) + 2 * e.roll(2, 1)
    layer.norm = torch.ones_like(layer.norm)
    layer.router = torch.nn.functional.one_hot(torch.arange(12, device="cuda"), 512).to(dtype)
    x = torch.zeros(12, 512, device="cuda", dtype=dtype)
    x[:, :12] = part.to(dtype)
    assert layer.routing_changes(x, r[:12]) == 0
    layer.router = torch.randn(12, 512, generator=g, device="cuda").to(dtype) / 20
    x = torch.randn(200, 512, generator=g, device="cuda").to(dtype)
    _, n, rounded = layer.normalised(x, r)
    logits = n @ layer.router.double().t()
    kept = 0
    for t in range(200):
        best = set(sorted(range(12), key=lambda i: -logits[t, i].item())[:3])
        kept += len(best & set(layer.chosen(rounded)[t].tolist()))
    assert layer.routing_changes(x, r) == pytest.approx(1 - kept / 600, abs=1e-12)
    layer.chosen = lambda rows: torch.full((200, 3), 5, device="cuda") + torch.arange(3, device="cuda") * (
        1 if rows.dtype == torch.float64 else -1)
    assert layer.routing_changes(x, r) == pytest.approx(2 / 3)      # 5, 6, 7 and 5, 4, 3 share one
