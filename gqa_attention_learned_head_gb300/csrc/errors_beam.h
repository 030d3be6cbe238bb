// errors_beam.h -- the error word's bits that only the beam step's kernels raise; as those of ptx.cuh, bit i is status
// code i of include/sinkattn.h.  Internal to libsinkattn.
#pragma once

namespace sinkattn {

enum : unsigned {
    kErrNoPages = 1u << 8,
    kErrBadValue = 1u << 9,
    kErrBadIndex = 1u << 10,
};

}  // namespace sinkattn
