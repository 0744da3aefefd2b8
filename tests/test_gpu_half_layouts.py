"""The lane layouts that the 16-bit kernels assume (half_types.hpp), pinned on
the device one instruction at a time: both matrix instructions in both types,
the transposing LDS read, the exchange between 16-lane rows and the two-byte
loads into LDS.  Each output
is compared with the plain definition computed on the host."""
import ctypes
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

PROBES = os.path.join(os.path.dirname(os.path.abspath(__file__)), "hip", "libhalf_layout_probes.so")
TYPES = [(0, torch.float16), (1, torch.bfloat16)]


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if not os.path.exists(PROBES):
        raise RuntimeError(f"{PROBES} is missing: run __graft_entry__.build()")
    lib = ctypes.CDLL(PROBES)
    for name in ("probe_mfma32", "probe_mfma16", "probe_read_transposed", "probe_transpose_rows", "probe_dma2"):
        getattr(lib, name).argtypes = [ctypes.c_int] + [ctypes.c_void_p] * 4
        getattr(lib, name).restype = ctypes.c_int
    return lib


def _call(f, kind, *tensors):
    assert f(kind, *[t.data_ptr() for t in tensors], torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind,dtype", TYPES)
@pytest.mark.parametrize("name,rows,k", [("probe_mfma32", 32, 16), ("probe_mfma16", 16, 32)])
def test_matrix_instruction_layout(lib, name, rows, k, kind, dtype):
    g = torch.Generator().manual_seed(rows + kind)
    # small integers: every product and sum is exact
    a = torch.randint(-15, 16, (rows, k), generator=g).to(dtype)
    b = torch.randint(-15, 16, (rows, k), generator=g).to(dtype)
    c = torch.full((rows, rows), float("nan"), device="cuda")
    _call(getattr(lib, name), kind, a.cuda(), b.cuda(), c)
    assert torch.equal(c.cpu(), a.float() @ b.float().t())


def test_transposing_read(lib):
    values = torch.arange(512, dtype=torch.int16)
    rng = np.random.default_rng(3)
    addr = torch.from_numpy(rng.permutation(128)[:64].astype(np.int32) * 8)     # any 8-byte places
    out = torch.zeros(64, 4, dtype=torch.int16, device="cuda")
    _call(lib.probe_read_transposed, 0, values.cuda(), addr.cuda(), out)
    want = torch.empty(64, 4, dtype=torch.int16)
    for lane in range(64):
        group, c = lane // 16 * 16, lane % 16
        for b in range(4):
            source = addr[group + 4 * b + c // 4].item() // 2 + c % 4
            want[lane, b] = values[source]
    assert torch.equal(out.cpu(), want)


def test_exchange_between_lane_rows(lib):
    words = torch.arange(256, dtype=torch.int32).reshape(64, 4)
    out = torch.zeros(64, 4, dtype=torch.int32, device="cuda")
    _call(lib.probe_transpose_rows, 0, words.cuda(), torch.zeros(64, dtype=torch.int32, device="cuda"), out)
    rows = words.reshape(4, 16, 4)                   # row, lane of the row, word
    assert torch.equal(out.cpu().reshape(4, 16, 4), rows.permute(2, 1, 0))


def test_two_byte_loads_into_lds(lib):
    """Lane l's value lands in word l, zero-extended; behind the records, zeros."""
    values = torch.arange(1000, 1128, dtype=torch.int16)
    g = torch.Generator().manual_seed(2)
    offset = 2 * torch.randint(0, 128, (64,), generator=g).int()
    offset[5], offset[40], offset[63] = 256, 4096, -2 ** 31      # out of range
    out = torch.zeros(64, dtype=torch.int32, device="cuda")
    _call(lib.probe_dma2, 0, values.cuda(), offset.cuda(), out)
    want = torch.where((offset >= 0) & (offset < 256), values[(offset.clamp(0, 254) // 2).long()].int(), 0)
    assert torch.equal(out.cpu(), want)
