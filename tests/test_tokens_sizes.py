"""Sizes that a token-level call does not take are refused as such, before
anything is allocated for them, with and without tokens.  The checks run here
on host tensors: what looks for a device is put aside, and nothing gets past
the library's own refusal."""
import os

import pytest
import torch

import mxfp8_block_scaled_05_amd as m
from mxfp8_block_scaled_05_amd import logprobs, moe


@pytest.fixture
def host(monkeypatch):
    if not os.path.exists(m.LIB_PATH):
        pytest.skip("libmxfp8.so not built")
    if torch.cuda.is_available():
        pytest.skip("passes host memory")
    for mod in (moe, logprobs):
        monkeypatch.setattr(mod, "need", lambda t, dtype, name: t.data_ptr())
        monkeypatch.setattr(mod, "need_rows", lambda t, name: (0, t.shape[1]))
        monkeypatch.setattr(mod, "same_device", lambda *t: 0)
        monkeypatch.setattr(mod, "stream_of", lambda dev: None)


@pytest.mark.parametrize("T", [0, 3])
@pytest.mark.parametrize("k", [-1, 0, 9, 33, 1 << 40])
def test_route(host, T, k):
    with pytest.raises(m.MXFP8Error, match="mxfp8_route: MXFP8_ERR_SHAPE"):
        m.route(torch.zeros(T, 8), k)


@pytest.mark.parametrize("T", [0, 3])
@pytest.mark.parametrize("experts,pad,rows", [(0, 32, None), (-5, 32, None), (1025, 32, None), (8, 0, None), (8, -32, None),
                                              (8, 1025, None), (8, 32, -1), (1 << 40, 32, None), (8, 32, 1 << 31), (8, 32, 1 << 45)])
def test_route_tables(host, T, experts, pad, rows):
    with pytest.raises(m.MXFP8Error, match="mxfp8_route_tables: MXFP8_ERR_SHAPE"):
        m.route_tables(torch.zeros((T, 2), dtype=torch.int32), experts, pad, rows)


def test_route_tables_without_tokens(host):
    t = m.route_tables(torch.zeros((0, 2), dtype=torch.int32), 8, 128, rows=256)
    assert t.offsets.tolist() == [0] * 9 and t.counts.tolist() == [0] * 8 and t.row_token.tolist() == [-1] * 256
    assert t.pair_row.shape == (0, 2) and t.pad == 128


@pytest.mark.parametrize("T", [0, 3])
@pytest.mark.parametrize("n", [-1, 9, 65, 1 << 40])
def test_token_logprobs(host, T, n):
    with pytest.raises(m.MXFP8Error, match="mxfp8_token_logprobs: MXFP8_ERR_SHAPE"):
        m.token_logprobs(torch.zeros(T, 8), torch.zeros(T, dtype=torch.int64), top_n=n)
