"""Histories of more than 8192 tokens over vocabularies of several CTAs: each CTA of a row reads its share and tells the owners of
the tokens, in each of the kernel's forms (few rows: 1024 threads a CTA; many: 512; 32- and 64-bit tokens; rows aligned to 16
bytes or not), bit for bit as plain fp32 arithmetic."""
import numpy as np
import pytest
import torch

import q8_block_quantized_gemv_gb300 as q8
from test_gpu_choose import built, everything, logits_of, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("m,N,width", [(2, 20000, 8193), (3, 2049, 9001), (24, 20000, 8200), (40, 16385, 12001), (80, 5000, 8500),
                                       (33, 32003, 9999), (21, 400000, 8300)])
def test_shared_histories(m, N, width, wide):
    """Rows of more and of fewer than 8192 tokens beside each other; some of no tokens at all."""
    rules = everything(m, N, width, seed=m + N, wide=wide)
    rules["lengths"][1::4] = width
    for i, r in enumerate(range(2, m, 3)):
        rules["lengths"][r] = (8192, 8193, 0, 1, 5000, 8191, 8194)[i % 7]
    rules["prompts"] = np.where(np.arange(m) % 3 == 0, rules["lengths"] - 7, rules["lengths"] // 3).astype(np.int32)
    rules["history"][0, ::3] = N - 1  # the last CTA's, from every share
    run(logits_of(m, N, m), **rules)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("width", [131073, 1048575])
def test_one_token_fills_a_history(width, wide):
    """A count near the end of its field, made by the atomics of eight CTAs; the prompt ends inside another CTA's share."""
    m, N = 3, 20000
    rules = everything(m, N, width, seed=width % 1000, wide=wide)
    rules["history"][0, :] = 19999
    rules["history"][1, 100:] = 2
    rules["lengths"][:] = [width, width - 3, width]
    rules["prompts"][:] = [0, width // 8 * 3 + 5, width - 2]
    rules["frequency"][:] = [1e-3, 3e-4, 0.5]
    run(logits_of(m, N, 5), **rules)


@pytest.mark.parametrize("m", [4, 30])
def test_tokens_outside_the_vocabulary(m):
    N, width = 20000, 8600
    rules = everything(m, N, width, seed=m)
    h = rules["history"]
    h[:, ::5], h[:, 1::7], h[:, 2::9] = -1, N, 2 ** 31 - 1
    rules["lengths"][:] = width + 100
    run(logits_of(m, N, 6), **rules)
    wide = dict(rules, history=h.astype(np.int64))
    wide["history"][:, 3::11], wide["history"][:, 4::11] = 2 ** 32 + 5, -2 ** 40 + 6
    run(logits_of(m, N, 6), **wide)


def test_in_place_over_several_turns():
    """A vocabulary of more than eight slices: the words are made anew for each turn, the history read again."""
    m, N, width = 20, 400003, 8500
    rules = everything(m, N, width, seed=9, wide=True)
    rules["lengths"][:] = width
    run(logits_of(m, N, 7), place=True, **rules)
