// host_device.h — functions that kernels run and host tests compile.
#pragma once

#ifdef __CUDACC__
#define BGQ_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define BGQ_HOST_DEVICE inline
#endif
