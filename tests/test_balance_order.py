"""How the balance loss's blocks hand their terms to the last one, in the compiled device
code (CPU only). The stores of a block's results and the count behind them are relaxed
atomics at agent scope with a wait between them, which the language does not order: the
instructions have to be the ones that order it. Stores and loads go past the caches that
blocks do not share (sc1), all stores have completed before the count goes out, and what is
read after the count is read past those caches, too."""
import os
import re
import subprocess

import pytest

from combine_ep_layout_10_amd import build as B


@pytest.fixture(scope="module")
def body(tmp_path_factory):
    if not os.path.exists(B.HIPCC):
        pytest.skip("hipcc not installed")
    out = tmp_path_factory.mktemp("route") / "route.s"
    flags = [f for f in B.FLAGS if f not in ("-shared", "-fPIC")]
    subprocess.run([B.HIPCC] + flags + ["--cuda-device-only", "-S", "-o", str(out), os.path.join(B.CSRC, "ep_route.hip")],
                   check=True, capture_output=True)
    text = re.search(r"^(_ZN2ep\w*k_balance_loss\w*):.*?^\.Lfunc_end", out.read_text(), re.M | re.S).group(0)
    lines = [l.split(";")[0].strip() for l in text.splitlines()]
    return [l for l in lines if l]


def handover(lines):
    """What is wrong with the order of a block's results, its count and the last block's loads."""
    wrong = []
    counts = [i for i, l in enumerate(lines) if l.startswith("global_atomic_add ")]
    if len(counts) != 1 or not re.search(r"\bsc0\b", lines[counts[0]]):
        return ["one count that returns its value"]
    n = counts[0]
    passed = [i for i, l in enumerate(lines[:n]) if l.startswith("global_store_") and re.search(r"\bsc1\b", l)]
    if len(passed) != 2:
        wrong.append("a term and a number of tokens, past the caches")
    else:
        stores = [i for i, l in enumerate(lines[:n]) if re.match(r"(global|flat|buffer)_store_", l)]
        waits = [i for i, l in enumerate(lines[:n]) if l.startswith("s_waitcnt") and "vmcnt(0)" in l]
        if not waits or waits[-1] < stores[-1]:
            wrong.append("a wait for all stores before the count")
    loads = [l for l in lines[n:] if re.match(r"(global|flat|buffer)_load_", l)]
    if len(loads) < 2 or any(not re.search(r"\bsc1\b", l) for l in loads):
        wrong.append("loads past the caches after the count")
    if not any(l.startswith("s_barrier") for l in lines[n:]):
        wrong.append("a barrier after the count")
    return wrong


def test_results_complete_before_the_count(body):
    assert handover(body) == []


def test_a_missing_wait_or_a_plain_access_is_seen(body):
    """The check itself, on text that lacks what it looks for."""
    n = next(i for i, l in enumerate(body) if l.startswith("global_atomic_add "))
    last = max(i for i, l in enumerate(body[:n]) if l.startswith("global_store_"))
    assert handover(body[:last + 1] + [l for l in body[last + 1:n] if "vmcnt(0)" not in l] + body[n:])
    for i in range(len(body)):
        if re.search(r"^global_(load|store)_\w+ .*\bsc1\b", body[i]):
            assert handover(body[:i] + [re.sub(r" sc1\b", "", body[i])] + body[i + 1:]), body[i]
