"""Orders inside the kernels that no run is to try, read from the sources (no GPU needed)."""
import os
import re

import pytest

import mixture_experts_lora_b200 as ml

CSRC = os.path.join(os.path.dirname(os.path.abspath(ml.__file__)), "csrc")


def kernels():
    """(file, name, body) of every kernel, comments taken out."""
    out = []
    for f in sorted(os.listdir(CSRC)):
        src = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(os.path.join(CSRC, f)).read(), flags=re.S)
        for m in re.finditer(r"__global__", src):
            at = src.index("{", m.end())
            name = re.findall(r"(\w+_kernel)\s*\(", src[m.end():at])[0]
            depth, end = 1, at + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(src[end], 0)
                end += 1
            out.append((f, name, src[at:end]))
    return out


KERNELS = kernels()


def test_all_kernels_are_found():
    names = {n for _, n, _ in KERNELS}
    assert {"lora_tiles_kernel", "lora_single_kernel", "rank_r_kernel", "adamw_kernel", "balance_sum_kernel"} <= names
    assert sum(re.search(r"tmem_alloc", b) is not None for _, _, b in KERNELS) >= 5


@pytest.mark.parametrize("f,name,body", KERNELS, ids=[n for _, n, _ in KERNELS])
def test_dependents_are_let_in_once_tmem_is_held(f, name, body):
    """A dependent may hold TMEM columns while it waits for the grid before it: that grid's CTAs hold
    theirs before they let it in."""
    take = [m.start() for m in re.finditer(r"\btmem_alloc\w*\(", body)]
    let = [m.start() for m in re.finditer(r"\b(pdl_begin|pdl_launch_dependents)\(", body)]
    assert len(let) == 1, f"{f}: {name}"
    assert all(t < let[0] for t in take), f"{f}: {name}"


def test_shared_memory_stores_are_fenced_before_a_bulk_copy_overwrites_them():
    """lora_tiles_kernel: the warps that have stored into a slot of rows hand it to the loader, whose copy
    goes through another proxy: a fence stands between, in every branch."""
    body = next(b for _, n, b in KERNELS if n == "lora_tiles_kernel")
    parts = body[body.index("= pack8(y)"):].split("mbar_arrive(smem_u32(&yfree[st]))")
    assert len(parts) == 3
    assert all("fence_proxy_async_smem()" in p for p in parts[:2])
