"""Partitioned on-chip (LDS) integer histogram for AMD Instinct MI355X (gfx950).

``hist.Plan`` / ``hist.run`` call the C-ABI library libpca_hist.so, whose HIP
kernels do all of the work; ``experts`` holds the operators of a mixture-of-experts layer;
``inputs`` draws the seeded synthetic workloads.
"""
from . import experts, hist  # noqa: F401
from .hist import Plan, run  # noqa: F401
