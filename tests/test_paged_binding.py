"""What the paged calls' binding refuses before the library is called; the library's entries are stubs here that note a call."""
import subprocess
import sys
import types

import pytest
import torch

from ultra_long_context_b200 import hsa

BF16 = torch.bfloat16


@pytest.fixture
def calls(monkeypatch):
    made = []

    def entry(name):
        return lambda *a: made.append((name, a)) or 0

    names = ("hsa_page_plan", "hsa_page_append", "hsa_prefix_decode")
    monkeypatch.setattr(hsa, "_lib", types.SimpleNamespace(**{n: entry(n) for n in names}))
    monkeypatch.setattr(hsa, "_stream_of", lambda dev, stream: 0)
    return made


def decode_args(B=2, H=2, Hkv=1, D=64, pages=3, npre=1, width=2, device="cpu"):
    pool = torch.zeros(2, pages, Hkv, 64, D, dtype=BF16, device=device)
    return (torch.zeros(B, H, D, dtype=BF16, device=device), pool[0], pool[1], torch.zeros(npre, dtype=torch.int32, device=device),
            torch.zeros(1, dtype=torch.int64, device=device), torch.zeros(B, width, dtype=torch.int32, device=device),
            torch.zeros(B, dtype=torch.int64, device=device))


@pytest.mark.parametrize("workspace,error", [
    (torch.empty(1 << 16, dtype=torch.uint8, device="meta"), ValueError),     # another device
    (torch.empty(1 << 16, 2, dtype=torch.uint8)[:, 0], ValueError),            # a view with gaps
    (1 << 20, TypeError),
])
def test_prefix_decode_refuses_a_workspace_that_it_cannot_use(calls, workspace, error):
    with pytest.raises(error, match="workspace"):
        hsa.hsa_prefix_decode(*decode_args(), workspace=workspace)
    assert not calls
    hsa.hsa_prefix_decode(*decode_args(), workspace=torch.empty(1 << 16, dtype=torch.uint8))
    assert [n for n, _ in calls] == ["hsa_prefix_decode"]


@pytest.mark.parametrize("args", [
    (8192, 1 << 27, 1 << 17, 128, 8, 8),         # 2^32 row groups
    (8192, 1 << 17, 1 << 17, 128, 8, 8), (64, 8, 8, 128, 1 << 24, 8), (1, 8, 8, 128, 8, 1 << 24), (128, 8, 8, 128, 8, 1 << 23),
])
def test_prefix_decode_workspace_size_is_zero_for_sizes_that_the_call_refuses(args):
    """In a process of its own: a division by zero would end it."""
    code = f"from ultra_long_context_b200 import hsa; print(hsa.hsa_prefix_decode_workspace_size(*{args}))"
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert run.returncode == 0 and run.stdout.strip() == "0", (run.returncode, run.stdout)


@pytest.mark.parametrize("kw,status", [
    (dict(ws=None), -3), (dict(ws=(1 << 20) + 16), -3), (dict(size=128), -3), (dict(limit=0), -1), (dict(limit=1000001), -1), (dict(after=1000001), -1),
])
def test_selftest_timed_wait_checks_its_arguments_on_host(kw, status):
    args = dict(ws=1 << 20, size=4096, limit=1000, after=1000, arrive=1, stream=None)
    args.update(kw)
    assert hsa.lib().hsa_selftest_timed_wait(*args.values()) == status and hsa.hsa_last_error() != ""


def meta(*shape, dtype):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("width,ring,tokens", [(4, 9, (1 << 32) + 5), (4, (1 << 32) + 9, 8), ((1 << 32) + 1, 9, 8), (4, 9, 1 << 31)])
def test_page_plan_refuses_sizes_past_32_bits(calls, width, ring, tokens):
    """The C call takes them as int: a larger one would arrive as another size."""
    with pytest.raises(ValueError, match="2\\^31"):
        hsa.hsa_page_plan(meta(2, dtype=torch.int64), meta(2, dtype=torch.int32), meta(2, width, dtype=torch.int32), meta(ring, dtype=torch.int32),
                          meta(3, dtype=torch.int64), tokens)
    assert not calls


def test_page_append_refuses_sizes_past_32_bits(calls):
    n, pages = (1 << 32) + 1, (1 << 32) + 3
    for n, pages in ((n, 3), (1, pages)):
        K, pool = meta(n, 1, 64, dtype=BF16), meta(pages, 1, 64, 64, dtype=BF16)
        with pytest.raises(ValueError, match="2\\^31"):
            hsa.hsa_page_append(K, K, meta(n, dtype=torch.int64), pool, pool)
    assert not calls


@pytest.mark.parametrize("kw", [dict(npre=1 << 32), dict(width=(1 << 32) + 1), dict(pages=(1 << 32) + 3)])
def test_prefix_decode_refuses_sizes_past_32_bits(calls, kw):
    def args(B=2, H=2, Hkv=1, D=64, pages=3, npre=1, width=2):
        pool = meta(pages, Hkv, 64, D, dtype=BF16)
        return (meta(B, H, D, dtype=BF16), pool, pool, meta(npre, dtype=torch.int32), meta(1, dtype=torch.int64),
                meta(B, width, dtype=torch.int32), meta(B, dtype=torch.int64))

    with pytest.raises(ValueError, match="2\\^31"):
        hsa.hsa_prefix_decode(*args(**kw), workspace=meta(1 << 20, dtype=torch.uint8))
    assert not calls
    hsa.hsa_prefix_decode(*args(), workspace=meta(1 << 20, dtype=torch.uint8))
    assert len(calls) == 1


def test_a_stream_of_another_device_is_refused(calls):
    """The call would have run on the tensors' device, on its current stream, in no order with the one that was asked for."""
    other = types.SimpleNamespace(device=torch.device("cuda:1"), cuda_stream=0)
    q, Kp, Vp, pre, plen, table, own = decode_args()
    K = torch.zeros(4, 1, 64, dtype=BF16)
    with pytest.raises(ValueError, match="stream"):
        hsa.hsa_prefix_decode(q, Kp, Vp, pre, plen, table, own, workspace=torch.empty(1 << 16, dtype=torch.uint8), stream=other)
    with pytest.raises(ValueError, match="stream"):
        hsa.hsa_page_append(K, K, torch.zeros(4, dtype=torch.int64), Kp, Vp, stream=other)
    with pytest.raises(ValueError, match="stream"):
        hsa.hsa_page_plan(own, own.int(), table, pre, torch.zeros(3, dtype=torch.int64), 4, stream=other)
    assert not calls
