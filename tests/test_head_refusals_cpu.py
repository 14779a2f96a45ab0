"""Pointers that pe_sample and pe_verify refuse before anything touches the
device: vectors that are not aligned to their elements."""

import os

import pytest

BASE = 1 << 20     # host addresses stand in for device pointers: a refused call reads none


@pytest.fixture(scope="module")
def lib():
    from speculative_drafting_expand_gb300 import binding, build
    if not os.path.exists(binding.LIB_PATH):
        build.build()
    return binding.lib()


SAMPLE = dict(rows=3, vocab=100, dtype=1, logits=BASE, stride=100, temperature=BASE, top_k=BASE,
              top_p=BASE, min_p=BASE, u=BASE, tokens=BASE, logprobs=BASE, dist=BASE, stream=0)
VERIFY = dict(B=2, T=5, vocab=100, dtype=1, logits=BASE, stride=100, ids=BASE, cu_in=BASE,
              temperature=BASE, top_k=BASE, top_p=BASE, min_p=BASE, accept_u=BASE, u=BASE,
              draft_logits=0, draft_stride=0, draft_dist=0, num_accepted=BASE, sampled_ids=BASE,
              logprobs=BASE, dist=BASE, err=BASE, stream=0)


@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("name", ["temperature", "top_k", "top_p", "min_p", "u", "tokens",
                                  "logprobs"])
def test_sample_refuses_misaligned_vectors(lib, name, off):
    assert lib.pe_sample(*dict(SAMPLE, **{name: BASE + off}).values()) == 1


@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("name", ["ids", "cu_in", "temperature", "top_k", "top_p", "min_p",
                                  "accept_u", "u", "num_accepted", "sampled_ids", "logprobs",
                                  "err"])
def test_verify_refuses_misaligned_vectors(lib, name, off):
    assert lib.pe_verify(*dict(VERIFY, **{name: BASE + off}).values()) == 1
