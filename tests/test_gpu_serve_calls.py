"""Calls of the serving operators that their documentation allows and single-call tests do not make:
streams that share the status word, steps that go back, lengths and hints at the ends of their range."""
import math

import pytest
import torch

import serve_ref as R

pytestmark = pytest.mark.gpu
PAGE = 16


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def status():
    from block_diffusion_drafter_forward_gb300 import serve_status
    return serve_status()


def test_the_status_word_is_read_and_cleared_at_once():
    """While one stream sets a bit all along and reads, another's bit arrives whenever it was set.  (A torch
    operation on the word would be a load and a store: bits set between them were lost.)"""
    from block_diffusion_drafter_forward_gb300 import PagedKV, _lib, extend_tables, serve
    status()
    word = serve._status[torch.cuda.current_device()]
    kv = PagedKV(torch.zeros(2, 1, 2, PAGE * 64, device="cuda"))
    one = torch.ones(1, 1, 64, device="cuda")
    bad = i32([2 * PAGE])
    version = word._version
    kv.append(one, one, bad)
    assert status() == _lib.DFLASH_DEV_BAD_PAGE and status() == 0
    assert word._version == version
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    full = (i32([0]), i32([1]), i32([[0]]), i32([0]), i32([1]), 1)
    for _ in range(100):
        kv.append(one, one, bad, stream=side)
        seen = 0
        for _ in range(3):
            extend_tables(*full)
            seen |= status()
        side.synchronize()
        assert seen | status() == _lib.DFLASH_DEV_BAD_PAGE | _lib.DFLASH_DEV_NO_ROOM
