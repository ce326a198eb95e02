// The plan behind eqconv_plan_t, and the checks that the entry points share.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <string>

#include "eqc_dispatch.h"
#include "eqc_tables.h"
#include "eqconv.h"

namespace eqc {

struct SymKernelSet;

// What a type embedding's or a block norm's plan holds beside C and device.
struct LayerSpec {
    bool norm;            // block norm (else embedding)
    int64_t V;            // embedding: rows of the table
    int64_t padding;      // embedding: the row without a gradient (-1: none)
    int in_type;          // element type codes of include/eqconv.h
    int out_type;
    int L, gate;          // block norm: degrees 0..L, gate function
    float eps;
};

// Records a CUDA failure for eqconv_last_error and gives its status.
int cuda_status(cudaError_t e, const char* where);
// EQCONV_OK when the plan's device is the current one.
int check_device(eqconv_plan_t plan);
// L of a natural-parity prefix "0e+1o+..." (-1 malformed, -2 another list).
int natural_prefix(const char* irreps);

inline bool aligned_to(const void* p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

}  // namespace eqc

struct eqconv_plan_s {
    int lin, lsh, lout, C;
    int fwd_vec, det_vec, atomic_vec;
    size_t gather_budget;   // bytes of gathered rows one band may touch (0: one band)
    bool budget_set;        // false: per-mode defaults (bands for the atomic backward only)
    int mode;               // output variant bits (eqc::kModeAllParity, eqc::kModePerPath)
    int P, D_in, D_sh, D_out;
    int paths[eqc::kMaxPaths][3];
    int path_rows[eqc::kMaxPaths];
    int device;
    unsigned* d_status;
    const eqc::KernelSet* fwd_ks;
    const eqc::KernelSet* det_ks;      // deterministic backward
    const eqc::KernelSet* atomic_ks;   // atomic backward
    const eqc::DblKernelSet* dbl_ks;   // double backward (summed natural-parity outputs only)
    bool node_product;                 // a node-local product plan (no convolution)
    const eqc::NpKernelSet* np_ks;     // node-local product
    const eqc::SymKernelSet* symc_ks;  // symmetric contraction (then node_product is true too)
    int n_species;
    const eqc::LayerSpec* layer;            // a type embedding or a block norm (then node_product is true too)
};
