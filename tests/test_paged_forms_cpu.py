"""More refusals of the torch helpers that need no GPU."""

import subprocess
import sys
import types

import pytest
import torch

import ulysses_sequence_gb300 as U

I32, BF16 = torch.int32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    from ulysses_sequence_gb300 import build
    build.build()
    return U.load()


def sized(*shape, dtype=I32):
    """A tensor of this size without memory."""
    return torch.empty(shape, dtype=dtype, device="meta")


FAKE = types.SimpleNamespace(device=-1, H_kv=1, d=64, ref=None)  # of a cache, where tensors without memory are


def test_helpers_refuse_tensors_past_32_bits():
    """The library's counts are 32-bit: a tensor with more tokens, requests, pages or list entries is refused, not taken by the
    low bits of its size (2^32 + 5 tokens would be five)."""
    n, one, table = 2 ** 32 + 5, sized(1), sized(1, 4)
    rows = sized(n, 1, 64, dtype=BF16)
    with pytest.raises(ValueError, match="32 bits"):
        U.kv_append(rows, rows, FAKE, sized(n))
    with pytest.raises(ValueError, match="32 bits"):
        U.paged_attn_fwd(rows, FAKE, sized(2), one, table)
    q = sized(1, 1, 64, dtype=BF16)
    with pytest.raises(ValueError, match="32 bits"):
        U.paged_attn_fwd(q, FAKE, sized(2), one, sized(1, n))
    with pytest.raises(ValueError, match="32 bits"):
        U.paged_attn_fwd(q, FAKE, sized(n + 1), sized(n), sized(n, 0))
    with pytest.raises(ValueError, match="32 bits"):
        U.page_plan(one, one, one, one, sized(1, n), 16, 10, 1)
    with pytest.raises(ValueError, match="32 bits"):
        U.page_plan(sized(n), sized(n), one, one, sized(n, 0), 16, 10, 1)
    with pytest.raises(ValueError, match="32 bits"):
        U.page_plan(one, one, sized(n), one, table, 16, 10, 1)
    for shape in ((n, 16, 1, 64), (1, 2 ** 32 + 16, 1, 64), (1, 16, n, 64), (1, 16, 1, 2 ** 32 + 64)):
        with pytest.raises(ValueError, match="32 bits"):
            U.PagedCache(sized(*shape, dtype=BF16), sized(*shape, dtype=BF16))


def test_helpers_refuse_tensors_of_too_few_dimensions():
    scalar, row = sized(dtype=BF16), sized(64, dtype=BF16)
    for k in (scalar, row):
        with pytest.raises(ValueError, match="k must be"):
            U.kv_append(k, k, FAKE, sized(1))
        with pytest.raises(ValueError, match="q must be"):
            U.paged_attn_fwd(k, FAKE, sized(2), sized(1), sized(1, 4))
        with pytest.raises(ValueError, match="q must be"):
            U.paged_attn_workspace(k, FAKE)
    for table in (sized(), sized(4), sized(1, 2, 3)):
        with pytest.raises(ValueError, match="block_table must be"):
            U.paged_attn_fwd(sized(1, 1, 64, dtype=BF16), FAKE, sized(2), sized(1), table)
        with pytest.raises(ValueError, match="block_table must be"):
            U.page_plan(sized(1), sized(1), sized(1), sized(1), table, 16, 10, 1)


_WITHOUT_PRIVATE_NAMES = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import ulysses_sequence_gb300 as U
i = torch.zeros(1, dtype=torch.int32)
try:
    U.page_plan(i, i, i, i, torch.zeros(1, 4, dtype=torch.int32), 16, 4, 1)
except ValueError as e:
    assert "CUDA" in str(e)
    print("refused")
"""


def test_helpers_need_no_private_names_of_torch():
    """Where a build of torch does not have the two short cuts that the helpers take, its public calls do."""
    r = subprocess.run([sys.executable, "-c", _WITHOUT_PRIVATE_NAMES], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "refused" in r.stdout, r.stdout + r.stderr
