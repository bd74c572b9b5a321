"""Kernels that refill LDS by DMA behind a barrier of their own (CPU only; read
from the device assembly of this repository's sources): a wave has its LDS reads
back before it reaches that barrier, whatever the compiler does with the
products that use them."""
import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

from speculative_sampling_verification_vocab_amd import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_reads_are_done_before_the_barrier(tmp_path):
    flags = [f for f in B.FLAGS if f not in ("-shared", "-fPIC")]
    srcs = [s for s in B.sources() if "block_barrier()" in open(s).read()]
    assert {os.path.basename(s) for s in srcs} >= {"sv_static.hip", "sv_headq.hip"}

    def listing(src):
        out = str(tmp_path / (os.path.basename(src) + ".s"))
        subprocess.check_call([B.HIPCC, *flags, "--cuda-device-only", "-S", "-I", os.path.join(ROOT, "include"),
                               "-o", out, src], stderr=subprocess.DEVNULL)
        return open(out).read()
    with ThreadPoolExecutor(2) as ex:
        for src, asm in zip(srcs, ex.map(listing, srcs)):
            own = [b for b in re.findall(r"#ASMSTART(.*?)#ASMEND", asm, re.S) if "s_barrier" in b]
            kernels = len(set(re.findall(r"^(_ZN\S*_kernel\S*):", asm, re.M)))
            assert kernels and len(own) >= 3, (src, kernels, len(own))
            for b in own:
                assert re.search(r"s_waitcnt lgkmcnt\(0\)\s+s_barrier", b), (src, b)
